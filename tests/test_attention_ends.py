"""The ends of the attention calls' ranges: the most streams, heads and workgroups, calls beside each other, the same
call twice, workspaces of the size that the library names, and what a call may not touch."""
import numpy as np
import pytest

import oracle
from tests.helpers import say, to_dev, to_np
from tests.test_gpu_attention import _bf16, _cache, _check, _dev16, _offsets, _strided, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


def test_more_workgroups_than_one_launch_has_threads_for(B):
    """65535 sequences of one token and 1024 heads: one key each, so that the output is its value."""
    import torch
    n, hq, d = 65535, 1024, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(n, hq, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    kv = torch.randn(n, 2, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    say("attention of", n * hq, "workgroups")
    o = B.attention(q, kv, kv, torch.arange(n + 1, device="cuda"))
    assert torch.equal(o.view(n, 2, hq // 2, d), kv[:, :, None].expand(-1, -1, hq // 2, -1))


def test_more_workgroups_than_one_launch_has_threads_for_with_a_key_head_each(B):
    """The same with as many key heads, whose rows share no workgroup."""
    import torch
    n, h, d = 65535, 1024, 8
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(n, h, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    say("attention of", n * h, "workgroups")
    assert torch.equal(B.attention(q, q, q, torch.arange(n + 1, device="cuda")), q)


@pytest.mark.parametrize("q8", [False, True])
def test_the_most_streams_take_a_step(B, q8):
    import torch
    n, h, d = 65535, 24, 16
    gen = torch.Generator(device="cuda").manual_seed(2)
    shape = (n, h, 16, d)
    pools = [torch.zeros(shape, device="cuda", dtype=torch.int8 if q8 else torch.bfloat16) for _ in range(2)]
    sc = {x: torch.zeros(shape[:3], device="cuda") if q8 else None for x in ("k_scale", "v_scale")}
    table = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)[:, None].contiguous()
    k = torch.randn(n, h, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    start = torch.randint(0, 16, (n,), device="cuda", generator=gen, dtype=torch.int32)
    say("write and step of", n, "streams")
    B.kv_write(k, k, *pools, table, start=start, **sc)
    back, _ = B.kv_read(*pools, table, torch.arange(n + 1, device="cuda"), n, start=start, **sc)
    assert q8 or torch.equal(back, k)
    start.zero_()
    B.kv_write(k, k, *pools, table, start=start, **sc)
    o = B.attention_step(k, *pools, table, start + 1, **sc)
    back, _ = B.kv_read(*pools, table, torch.arange(n + 1, device="cuda"), n, **sc)
    # one key of weight 1: its value, whose two terms and rounding to bf16 are that of the row read back
    assert torch.equal(o, back)


@pytest.mark.parametrize("nseq", [63, 64, 65, 5000])
def test_many_short_sequences(B, nseq):
    rng = np.random.default_rng(nseq)
    lengths = rng.integers(0, 4, nseq)
    keys = lengths + rng.integers(0, 3, nseq) * rng.integers(0, 2, nseq)
    off, koff, d = _offsets(lengths), _offsets(keys), 32
    q, k, v = _bf16(rng, (int(off[-1]), 2, d)), _bf16(rng, (int(koff[-1]), 1, d)), _bf16(rng, (int(koff[-1]), 1, d))
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True)
    _check(B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff)), want, 2.0 ** -8, d)
    table, npages = _table(rng, keys, 16)
    pools = [_dev16(np.zeros((npages, 1, 16, d), np.float32)) for _ in range(2)]
    B.kv_write(_dev16(k), _dev16(v), *pools, to_dev(table), offsets=to_dev(koff))
    for got, x in zip(B.kv_read(*pools, to_dev(table), to_dev(koff), int(koff[-1])), (k, v)):
        assert np.array_equal(to_np(got), x)


def test_the_same_call_gives_the_same_bits_and_calls_beside_each_other_too(B):
    """Shares of a query's keys are joined in one order, whatever ends first."""
    import torch
    rng = np.random.default_rng(3)
    lengths = [5000, 17, 3000]
    pages, scales, table, dev, sc = _cache(rng, lengths, 2, 128, 64, True)
    q, n, dtable = _dev16(_bf16(rng, (3, 6, 128))), to_dev(np.array(lengths, np.int32)), to_dev(table)
    off, koff = to_dev(_offsets([40, 3, 90])), to_dev(_offsets([4000, 3, 2000]))
    pq, pk, pv = (_dev16(_bf16(rng, (m, h, 128))) for m, h in ((133, 6), (6003, 2), (6003, 2)))

    def both():
        return (B.attention_step(q, *dev, dtable, n, **sc), B.attention(pq, pk, pv, off, k_offsets=koff))
    first = both()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(both())
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))


@pytest.mark.parametrize("nseq,hq,hkv,d,positions", [(1, 12, 4, 128, 2048), (3, 5, 1, 40, 960), (300, 8, 8, 64, 64), (1, 1, 1, 8, 65536)])
def test_calls_stay_inside_the_workspaces_whose_size_the_library_names(B, nseq, hq, hkv, d, positions):
    import torch
    rng = np.random.default_rng(d)
    lengths = np.minimum(rng.integers(1, 400, nseq), positions)
    page = 64
    pages, scales, table, dev, sc = _cache(rng, lengths, hkv, d, page, False, cols=positions // page)
    q = _bf16(rng, (nseq, hq, d))
    size = B.attention_step_workspace(nseq, hq, hkv, d, positions)
    buf = torch.full((size + 4096,), 77, device="cuda", dtype=torch.uint8)
    o = B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(lengths.astype(np.int32)), ws=buf[:size])
    assert torch.all(buf[size:] == 77)
    _check(o, oracle.attention_step(q, *pages, table, lengths, sizes=True), 2.0 ** -16, d)
    if nseq > 3:
        return
    qlen = np.minimum(lengths, 30)
    off, koff = _offsets(qlen), _offsets(lengths + positions // 2)
    total, total_k = int(off[-1]), int(koff[-1])
    q, k, v = _bf16(rng, (total, hq, d)), _bf16(rng, (total_k, hkv, d)), _bf16(rng, (total_k, hkv, d))
    size = B.attention_workspace(nseq, total, total_k, hq, hkv, d)
    buf = torch.full((size + 4096,), 77, device="cuda", dtype=torch.uint8)
    o = B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff), ws=buf[:size])
    assert torch.all(buf[size:] == 77)
    _check(o, oracle.attention(q, k, v, off, k_offsets=koff, sizes=True), 2.0 ** -8, d)
    with pytest.raises(ValueError, match="workspace"):
        B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff), ws=buf[:size - 1])


@pytest.mark.parametrize("lengths,keys", [([90], [6000]), ([2, 0, 33], [3000, 0, 5000])])
@pytest.mark.parametrize("more", [{}, {"window": 700}, {"window": 600, "prefix": 1000}, {"causal": False}, {"cap": 3.0, "slopes": True}],
                         ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("d", [64, 128, 200])
def test_shares_of_long_keys(B, lengths, keys, more, d):
    """Few queries behind many keys go in shares; some shares hold no key that a query sees."""
    from tests.test_gpu_attention import _mask
    rng = np.random.default_rng(sum(keys) + d)
    off, koff = _offsets(lengths), _offsets(keys)
    q = _bf16(rng, (int(off[-1]) + 3, 4, d), 1.5)
    k, v = (_bf16(rng, (int(koff[-1]), 2, d)) for _ in range(2))
    host, dev = _mask(more, rng, len(lengths), 4)
    n = int(off[-1])
    want = oracle.attention(q[:n], k, v, off, k_offsets=koff, sizes=True, **host)
    import torch
    out = torch.full((n + 3, 4, d), 7.0, device="cuda", dtype=torch.bfloat16)
    B.attention(_dev16(q), *_strided(k, v), to_dev(off), k_offsets=to_dev(koff), o_out=out, **dev)
    assert torch.all(out[n:] == 7.0)  # behind the last sequence
    _check(out[:n], want, 2.0 ** -8, d, host.get("slopes"), max(keys))


@pytest.mark.parametrize("d", [64, 128])
def test_keys_that_are_not_seen_have_no_part_in_shares(B, d):
    """As in one piece: v of a key behind the window, of another sequence, or of a later position is not finite."""
    rng = np.random.default_rng(d + 1)
    off, koff = _offsets([20, 9]), _offsets([5000, 3000])
    q, k, v = _bf16(rng, (29, 2, d)), _bf16(rng, (8000, 1, d)), _bf16(rng, (8000, 1, d))
    want = oracle.attention(q, k, v, off, k_offsets=koff, window=1500, sizes=True)
    v2 = v.copy()
    v2[100:3400] = np.inf     # in front of every query's window
    v2[4999] = np.nan         # the last key of sequence 0: its last query sees it
    v2[5000 + 2995, 0, 5] = -np.inf  # seen by the last five queries of sequence 1
    o = to_np(B.attention(_dev16(q), _dev16(k), _dev16(v2), to_dev(off), k_offsets=to_dev(koff), window=1500)).astype(np.float64)
    lost = np.zeros(o.shape, bool)
    lost[19] = True
    lost[24:29, :, 5] = True
    assert not np.isfinite(o[lost]).any()
    o[lost] = want[0][lost]
    _check(to_dev(o), want, 2.0 ** -8, d)


@pytest.mark.parametrize("keys", [3, 700, 3000])
def test_queries_without_keys_beside_values_that_are_not_finite(B, keys):
    """More queries than keys: the first see none and get zeros, whatever the others' keys hold."""
    rng = np.random.default_rng(keys)
    n, d = keys + 45, 64
    off, koff = _offsets([n]), _offsets([keys])
    q, k, v = _bf16(rng, (n, 1, d)), _bf16(rng, (keys, 1, d)), _bf16(rng, (keys, 1, d))
    v[0] = np.nan
    for window in (None, 2):
        o = to_np(B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff), window=window))
        assert not o[:45].any() and np.isnan(o[45]).all()
        assert window is None or np.isfinite(o[45 + window:]).all()


def test_keys_without_weight_and_one_key_alone(B):
    """One key: its value bit for bit, whatever the score. Far scores: the others' weights vanish."""
    rng = np.random.default_rng(77)
    for d in (8, 64, 128, 256):
        q, k, v = _bf16(rng, (90, 3, d), 30.0), _bf16(rng, (90, 1, d), 30.0), _bf16(rng, (90, 1, d))
        o = B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(_offsets([90])), window=1)
        assert np.array_equal(to_np(o), np.repeat(v, 3, axis=1))
        want = oracle.attention(q, k, v, _offsets([90]), scale=1.0, sizes=True)  # scores of some 900 sqrt(d)
        _check(B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(_offsets([90])), scale=1.0), want, 2.0 ** -8, d)


@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 24), (10, 2, 64), (9, 3, 128), (1024, 1, 8), (300, 2, 16), (33, 1, 256)])
@pytest.mark.parametrize("more", [{}, {"window": 9, "prefix": 7}, {"cap": 2.0, "slopes": True}, {"causal": False}],
                         ids=lambda m: "-".join(m) or "plain")
def test_any_number_of_heads_to_a_key_head(B, hq, hkv, d, more):
    """A workgroup's rows are queries with all their heads: its first and last query may have only some there."""
    from tests.test_gpu_attention import _mask
    rng = np.random.default_rng(hq + d)
    lengths, keys = ([1, 0, 40, 3], [70, 5, 40, 2]) if hq < 100 else ([1, 0, 3], [40, 5, 3])
    off, koff = _offsets(lengths), _offsets(keys)
    q = _bf16(rng, (int(off[-1]), hq, d), 1.5)
    k, v = (_bf16(rng, (int(koff[-1]), hkv, d)) for _ in range(2))
    host, dev = _mask(more, rng, len(lengths), hq)
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True, **host)
    o = B.attention(_dev16(q), *_strided(k, v), to_dev(off), k_offsets=to_dev(koff), **dev)
    _check(o, want, 2.0 ** -8, d, host.get("slopes"), max(keys))


def test_values_that_are_not_finite_and_heads_that_share_their_rows(B):
    """Only queries that see such a value have it, in every head."""
    rng = np.random.default_rng(8)
    off = _offsets([30])
    q, k, v = _bf16(rng, (30, 6, 32)), _bf16(rng, (30, 2, 32)), _bf16(rng, (30, 2, 32))
    want = oracle.attention(q, k, v, off, sizes=True)
    v2 = v.copy()
    v2[21, 1, 3] = np.nan     # key head 1: heads 3, 4 and 5
    o = to_np(B.attention(_dev16(q), _dev16(k), _dev16(v2), to_dev(off))).astype(np.float64)
    lost = np.zeros(o.shape, bool)
    lost[21:, 3:, 3] = True
    assert np.isnan(o[lost]).all()
    o[lost] = want[0][lost]
    _check(to_dev(o), want, 2.0 ** -8, 32)


@pytest.mark.parametrize("d,q8", [(16, False), (16, True), (72, False), (128, True), (256, False)])
def test_one_long_stream(B, d, q8):
    """More shares of one stream's keys than a wave has lanes, in a step and for few queries."""
    rng = np.random.default_rng(d)
    n = 40001
    pages, scales, table, dev, sc = _cache(rng, [n], 1, d, 64, q8)
    q, lengths = _bf16(rng, (1, 3, d)), np.array([n], np.int32)
    want = oracle.attention_step(q, *pages, table, lengths, k_scale=scales[0], v_scale=scales[1], sizes=True)
    _check(B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(lengths), **sc), want, 2.0 ** -16, d)
    if q8:
        return
    off, koff = _offsets([2]), _offsets([n])
    q, k, v = _bf16(rng, (2, 3, d)), _bf16(rng, (n, 1, d)), _bf16(rng, (n, 1, d))
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True)
    _check(B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff)), want, 2.0 ** -8, d)


@pytest.mark.parametrize("keys", [None, [90, 0, 2600]])
def test_rows_in_front_of_the_first_sequence(B, keys):
    """Offsets that begin behind row 0: the rows in front are no sequence's, and are left, in one piece and in shares."""
    import torch
    rng = np.random.default_rng(5)
    ahead, lengths = 150, [40, 0, 20]
    off = _offsets(lengths) + ahead
    koff = off if keys is None else _offsets(keys) + 7
    total, total_k = int(off[-1]) + 9, int(koff[-1]) + (9 if keys is None else 1)
    q, k, v = _bf16(rng, (total, 6, 64)), _bf16(rng, (total_k, 2, 64)), _bf16(rng, (total_k, 2, 64))
    inside = slice(ahead, int(off[-1]))
    want = oracle.attention(q[inside], k[koff[0]:], v[koff[0]:], off - ahead, k_offsets=koff - koff[0], sizes=True)
    out = torch.full((total, 6, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(off), k_offsets=to_dev(koff), o_out=out)
    assert torch.all(out[:ahead] == 7.0) and torch.all(out[off[-1]:] == 7.0)
    _check(out[inside], want, 2.0 ** -8, 64)
    table, npages = _table(rng, lengths, 16)
    pools = [torch.full((npages, 2, 16, 64), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    rows = _dev16(_bf16(rng, (total, 2, 64)))
    B.kv_write(rows, rows, *pools, to_dev(table), offsets=to_dev(off))
    assert int((pools[0] == 3.0).all(-1).sum()) == npages * 2 * 16 - 2 * sum(lengths)
    back = [torch.full((total, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    B.kv_read(*pools, to_dev(table), to_dev(off), total, k_out=back[0], v_out=back[1])
    for x in back:
        assert torch.equal(x[inside], rows[inside]) and torch.all(x[:ahead] == 5.0) and torch.all(x[off[-1]:] == 5.0)


def test_steps_and_prompts_of_many_shares_in_a_graph(B):
    """A captured step and prompt whose keys go in many shares, with workspaces of their own, replayed over new values."""
    import torch
    rng = np.random.default_rng(6)
    pages, scales, table, dev, sc = _cache(rng, [9000], 1, 64, 32, True)
    dtable, n = to_dev(table), to_dev(np.array([9000], np.int32))
    off, koff = to_dev(_offsets([5])), to_dev(_offsets([12000]))
    q, pq, pk, pv = (_dev16(_bf16(rng, (m, h, 64))) for m, h in ((1, 4), (5, 4), (12000, 2), (12000, 2)))

    def both():
        return B.attention_step(q, *dev, dtable, n, **sc), B.attention(pq, pk, pv, off, k_offsets=koff)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for length in (9000, 1, 0, 4321):
        n.fill_(length)
        q.copy_(_dev16(_bf16(rng, (1, 4, 64))))
        pq.copy_(_dev16(_bf16(rng, (5, 4, 64))))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, both()))


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 4), (128, 6, 2), (200, 4, 2)])
@pytest.mark.parametrize("more", [{}, {"prefix": 300}, {"cap": 4.0, "slopes": True}], ids=lambda m: "-".join(m) or "plain")
def test_many_blocks_of_ragged_prompts(B, d, hq, hkv, more):
    """Prompts whose blocks are taken in the order of their place, with empty and single ones among them, up to 63 of them."""
    from tests.test_gpu_attention import _mask
    rng = np.random.default_rng(d + hq)
    lengths = np.concatenate([[0, 900, 1, 0, 130, 128, 700, 0], rng.integers(0, 300, 54), [0]])
    assert len(lengths) == 63
    off = _offsets(lengths)
    q, k, v = (_bf16(rng, (int(off[-1]), h, d)) for h in (hq, hkv, hkv))
    host, dev = _mask(more, rng, len(lengths), hq)
    want = oracle.attention(q, k, v, off, sizes=True, **host)
    _check(B.attention(_dev16(q), *_strided(k, v), to_dev(off), **dev), want, 2.0 ** -8, d, host.get("slopes"), 900)
