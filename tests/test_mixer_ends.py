"""The mixer block's operators at their ends: rows without one finite value, sizes past one launch's
limits, and the bits that the states keep."""
import numpy as np
import pytest

import oracle
from synthdata import bf16_round
from tests.helpers import to_dev, to_np, say


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


# ---------------------------------------------------------------- 8-bit rows that hold a NaN or an infinity

def _lost_rows(d):
    """(x, w, lost): rows of d values, which of them have no finite 8-bit form.  w is NaN nowhere; its last entry is 0."""
    rng = np.random.default_rng(d)
    x = rng.standard_normal((10, d)).astype(np.float32)
    w = np.ones(d, np.float32)
    w[-1] = 0.0
    x[1] = np.nan                       # nothing but NaN
    x[2] = 0.0; x[2, 3] = np.nan        # NaN and zeros
    x[3] = -np.inf
    x[4, d // 2] = np.nan
    x[5] = 0.0; x[5, 1] = np.inf
    x[6, -1] = np.inf                   # under a weight of 0
    x[7] = 1e-35; x[7, 0] = np.nan      # beside values that alone would become zeros
    x[8] = 0.0
    lost = np.array([False] + [True] * 7 + [False] * 2)
    return x, w, lost


@pytest.mark.parametrize("d", [8, 64])
def test_oracle_rows_that_are_not_finite_have_no_finite_scale(d):
    x, w, lost = _lost_rows(d)
    with np.errstate(all="ignore"):
        _, plain = oracle.quant_rows_q8(x)
        _, scale, _ = oracle.rmsnorm_q8(x, w, 1e-6)
        _, by_weight, _ = oracle.rmsnorm_q8(np.ones((2, d)), np.where(np.arange(d) == 2, np.nan, 1.0), 1e-6)
    assert np.array_equal(~np.isfinite(plain), lost) and np.array_equal(~np.isfinite(scale), lost)
    assert plain[8] == 0 and scale[8] == 0
    assert not np.isfinite(by_weight).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [8, 64, 256, 512, 1024, 2048, 4096, 16384, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_not_finite_have_no_finite_scale(B, d, dtype):
    """Each width has its split of a row over threads, the last its second pass over memory."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    say("rows not finite", d, dtype)
    x, w, lost = _lost_rows(d)
    x = bf16_round(x)
    dx, dw = to_dev(x, dt), to_dev(w, dt)
    q, scale = B.quant_rows_q8(dx)
    assert np.array_equal(~np.isfinite(to_np(scale)), lost)
    q_o, step = oracle.quant_rows_q8(x[~lost])
    assert np.array_equal(to_np(q)[~lost], q_o) and np.array_equal(to_np(scale)[~lost] == 0, step == 0)
    q, scale, _ = B.rmsnorm_q8(dx, dw)
    assert np.array_equal(~np.isfinite(to_np(scale)), lost)
    q_o, _, _ = oracle.rmsnorm_q8(x[~lost], w, 1e-6)
    assert np.array_equal(to_np(q)[~lost], q_o)
    # split between x and the residual, many rows (another split of the row)
    half = torch.zeros_like(dx)
    half[:, ::2] = dx[:, ::2]
    _, scale, _ = B.rmsnorm_q8(half.repeat(500, 1), dw, residual=(dx - half).nan_to_num(0.0, 0.0, 0.0).repeat(500, 1))
    even = ~np.isfinite(x[:, ::2]).all(1)
    assert np.array_equal(~np.isfinite(to_np(scale)).reshape(500, 10), np.tile(even, (500, 1)))
    # a weight alone
    for bad in (np.nan, np.inf):
        w2 = np.ones(d, np.float32)
        w2[d // 2 + 1] = bad
        _, scale, _ = B.rmsnorm_q8(torch.ones(3, d, dtype=dt, device="cuda"), to_dev(w2, dt))
        assert not np.isfinite(to_np(scale)).any()


@pytest.mark.gpu
def test_nan_reaches_the_rows_behind_a_block(B):
    """A row lost in one product stays lost through the next norm and product."""
    import torch
    rng = np.random.default_rng(2)
    d = 128
    w8, ws = B.quant_rows_q8(to_dev(rng.standard_normal((d, d)).astype(np.float32)))
    x = torch.randn(5, d, device="cuda").to(torch.bfloat16)
    x[3] = float("nan")
    for _ in range(3):
        q, s, _ = B.rmsnorm_q8(x, torch.ones(d, device="cuda", dtype=torch.bfloat16))
        x = B.linear_i8(q, s, w8, ws)
    assert torch.isnan(x[3]).all() and torch.isfinite(x[[0, 1, 2, 4]]).all()


# ---------------------------------------------------------------- more rows than one launch has threads for

def _room(gigabytes):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of free GPU memory")


@pytest.mark.gpu
def test_rows_past_the_threads_of_a_launch(B):
    """2^28 rows of part of a wave each: every row right, the last ones among them."""
    import torch
    rows, d = (1 << 28) + 21, 8
    say("rows", rows, d)
    _room(16)
    top = (torch.arange(rows, device="cuda", dtype=torch.int32) % 119 + 9).to(torch.bfloat16)
    x = top[:, None].repeat(1, d)
    x[:, 3] = 0.0
    q, scale = B.quant_rows_q8(x)
    want = torch.full((d,), 127, dtype=torch.int8, device="cuda")
    want[3] = 0
    assert all(bool((part == want).all()) for part in q.split(1 << 26))
    # the scale as the type of one row gives it, for each of its 119 values
    few, s_few = B.quant_rows_q8(x[:119].contiguous())
    at = torch.arange(rows, device="cuda", dtype=torch.int32) % 119
    assert all(bool((a == s_few[b.long()]).all()) for a, b in zip(scale.split(1 << 26), at.split(1 << 26)))
    np.testing.assert_allclose(to_np(s_few), to_np(top[:119]) / 127.0, rtol=2.0 ** -23)


@pytest.mark.gpu
def test_wide_rows_past_the_threads_of_a_launch(B):
    """2^22 rows of a workgroup of 1024 each, in place."""
    import torch
    rows, d = (1 << 22) + 3, 8200
    say("rows", rows, d)
    dt = torch.bfloat16
    _room(rows * d * 2 / 1e9 + 8)
    rng = np.random.default_rng(d)
    some = bf16_round(rng.standard_normal((6, d)).astype(np.float32))
    at = [0, 1, (1 << 22) - 2, (1 << 22) - 1, rows - 2, rows - 1]
    w = torch.ones(d, dtype=dt, device="cuda")
    y_o, _ = B.rmsnorm(to_dev(some, dt), w)
    x = torch.zeros(rows, d, dtype=dt, device="cuda")
    for i, r in enumerate(at):
        x[r] = to_dev(some[i], dt)
    y, _ = B.rmsnorm(x, w, y_out=x)
    for i, r in enumerate(at):
        assert torch.equal(y[r], y_o[i])
    assert not y[2:2000].any() and not y[(1 << 22) - 2000:(1 << 22) - 2].any()


@pytest.mark.gpu
def test_channels_past_the_threads_of_a_launch(B):
    """2^28 output channels of a product of few tokens."""
    import torch
    m, n, k = 2, (1 << 28) + 41, 16
    say("channels", m, n, k)
    _room(24)
    gen = torch.Generator(device="cuda").manual_seed(4)
    wq = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda", generator=gen)
    xq = torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda", generator=gen)
    sx = torch.tensor([1.0, 0.5], device="cuda")
    y = B.linear_i8(xq, sx, wq, torch.ones(n, device="cuda"), out_dtype=torch.float32)
    for a in range(0, n, 1 << 24):  # sums below 2^24: exact in fp32
        b = min(a + (1 << 24), n)
        assert torch.equal(y[:, a:b], (xq.float() @ wq[a:b].float().t()) * sx[:, None])


@pytest.mark.gpu
def test_heads_past_the_threads_of_a_launch(B):
    """Short sequences whose heads and columns need more workgroups than one launch has along x: the last
    sequences equal those computed alone, and the oracle's."""
    import torch
    nseq, tokens, hv, dk, dv = 8192, 7, 65, 8, 1024
    say("heads", nseq, tokens, hv, dk, dv)
    _room(60)
    n, bf = nseq * tokens, torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k = (torch.randn(n, 1, dk, device="cuda", dtype=bf, generator=gen) for _ in range(2))
    v = torch.randn(n, hv, dv, device="cuda", dtype=bf, generator=gen)
    g = -0.2 * torch.rand(n, hv, device="cuda", generator=gen)
    beta = torch.rand(n, hv, device="cuda", generator=gen)
    off = torch.arange(nseq + 1, device="cuda") * tokens
    o = torch.full((n, hv, dv), float("nan"), device="cuda", dtype=bf)
    B.gated_delta(q, k, v, g, beta, off, want_state=False, o_out=o)
    few = 128
    for first in (0, nseq - few):
        rows = slice(first * tokens, (first + few) * tokens)
        alone, _ = B.gated_delta(q[rows], k[rows], v[rows], g[rows], beta[rows], off[:few + 1], want_state=False)
        assert torch.equal(o[rows], alone)
    assert all(bool(torch.isfinite(part).all()) for part in o.split(4096))
    last = slice(n - tokens, n)
    o_o, _ = oracle.gated_delta(*(to_np(t[last]) for t in (q, k, v, g, beta)), np.array([0, tokens]),
                                scale=dk ** -0.5, unit_qk=True)
    # one rounding to bf16 (within 2^-8 of an element) beside operands of 16 bits
    err = np.linalg.norm(to_np(o[last]) - o_o, axis=2) / np.linalg.norm(o_o, axis=2)
    assert err.max() <= 2.0 ** -8


# ---------------------------------------------------------------- the norm's divisor

@pytest.mark.gpu
def test_the_norms_divisor_is_rounded_once(B):
    """Rows whose mean square is exact in fp32, with a first value and weight of 1: y there is the divisor
    itself, within half a unit in the last place (and 1 % of one for the correction's own arithmetic)."""
    i, j = np.meshgrid(np.arange(128), np.arange(128))
    x = np.zeros((128 * 128, 4), np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, i.ravel() / 64.0, j.ravel() / 64.0
    y, _ = B.rmsnorm(to_dev(x), to_dev(np.ones(4, np.float32)), eps=0.0)
    r = to_np(y)[:, 0]
    want = 1.0 / np.sqrt(np.sum(x.astype(np.float64) ** 2, axis=1) / 4.0)
    assert np.max(np.abs(r - want) / np.spacing(want.astype(np.float32))) <= 0.51


@pytest.mark.gpu
def test_the_norms_divisor_at_its_ends(B):
    """Mean squares of zero, of subnormal numbers and past the largest number; eps alone."""
    x = np.zeros((5, 4), np.float32)
    x[1] = 1e-20
    x[2] = 1e20       # its square is infinite: zeros
    x[3] = 1e-22
    x[4, 0] = 2.0
    with np.errstate(all="ignore"):
        y = to_np(B.rmsnorm(to_dev(x), to_dev(np.ones(4, np.float32)), eps=0.0)[0])
    assert np.isnan(y[0]).all() and not y[2].any()
    np.testing.assert_allclose(y[1], 1.0, rtol=1e-4)  # 1e-40 has 17 bits
    np.testing.assert_allclose(y[4], [2.0, 0, 0, 0], rtol=2.0 ** -22)
    assert np.isfinite(y[3]).all() or np.isinf(y[3]).all()
    y = to_np(B.rmsnorm(to_dev(x), to_dev(np.ones(4, np.float32)), eps=1e-6)[0])
    np.testing.assert_allclose(y[1], 1e-20 * 1e3, rtol=2.0 ** -20)
    assert not y[0].any()


# ---------------------------------------------------------------- bits of the gated delta rule's state

# Every value of a state takes at most twelve fp32 roundings in a block: of K S0 and its product with the decay
# (3), the difference from V (1), U (3), its decay (2), the state's decay and sum (3).  Each is at most 2^-24 of its
# size, and what former blocks left fades with the state itself.  An operand on the state's way with 16 bits instead
# of 24 leaves 0.9e-6 to 1.5e-5 in these cases, whichever it is (K S0's S, the system's right side, its inverse, U).
STATE_BITS_TOL = 12 * 2.0 ** -24

BITS = [
    # few heads: four waves to 16 columns
    ([200, 130], 1, 2, 128, 64), ([300], 2, 2, 64, 64), ([250], 1, 1, 8, 16),
    # 32 and 64 columns a workgroup
    ([150, 200] * 8, 1, 8, 64, 64), ([129] * 8, 2, 8, 128, 128), ([100, 140] * 18, 2, 8, 64, 40), ([129] * 17, 2, 8, 128, 128),
    # long sequences of few heads in segments
    ([3000], 1, 2, 128, 128), ([1700], 1, 1, 64, 40), ([2600, 1900], 1, 1, 128, 32),
    # token by token
    ([5, 6, 4, 7], 2, 4, 128, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", BITS)
def test_gated_delta_state_keeps_24_bits(B, lengths, hk, hv, dk, dv, alike):
    """Keys of their own, and keys that share most of their direction, whose triangular system is far from one."""
    rng = np.random.default_rng(sum(lengths) + dk + dv)
    say("state bits", lengths[:4], hk, hv, dk, dv, alike)
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(off[-1])
    q, k = rng.standard_normal((2, n, hk, dk))
    if alike:
        k = k + 2.0 * rng.standard_normal((hk, dk))
    q, k = bf16_round(q.astype(np.float32)), bf16_round(k.astype(np.float32))
    v = bf16_round(rng.standard_normal((n, hv, dv)).astype(np.float32))
    g = (-0.05 * rng.random((n, hv)) ** 3).astype(np.float32)
    beta = rng.random((n, hv)).astype(np.float32)
    S0 = rng.standard_normal((len(lengths), hv, dk, dv)).astype(np.float32)
    _, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=dk ** -0.5, unit_qk=True, state=S0)
    import torch
    bf = torch.bfloat16
    _, S = B.gated_delta(to_dev(q, bf), to_dev(k, bf), to_dev(v, bf), to_dev(g), to_dev(beta), to_dev(off),
                         state_in=to_dev(S0))
    err = np.linalg.norm((to_np(S) - S_o).reshape(len(lengths) * hv, -1), axis=1)
    err /= np.linalg.norm(S_o.reshape(len(lengths) * hv, -1), axis=1)
    say("largest error", err.max())
    assert err.max() <= STATE_BITS_TOL


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hv,dk,dv", [([3000], 4, 128, 128), ([150, 0, 64] * 6, 8, 64, 64), ([90, 300] * 17, 8, 128, 128)])
def test_gated_delta_repeats_itself(B, lengths, hv, dk, dv):
    """The same call gives the same bits, beside other work and into memory that held something else."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    off = to_dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64))
    n, bf = sum(lengths), torch.bfloat16
    q, k, v = (torch.randn(n, hv, w, device="cuda", dtype=bf, generator=gen) for w in (dk, dk, dv))
    g, beta = -0.1 * torch.rand(n, hv, device="cuda", generator=gen), torch.rand(n, hv, device="cuda", generator=gen)
    o, S = B.gated_delta(q, k, v, g, beta, off)
    ws = torch.empty(B.gated_delta_workspace(len(lengths), n, hv, dk, dv), dtype=torch.uint8, device="cuda")
    for fill in (0, 0xFF, 0x3F):
        ws.fill_(fill)
        o2, S2 = torch.full_like(o, float("nan")), torch.full_like(S, float("nan"))
        B.gated_delta(q, k, v, g, beta, off, o_out=o2, state_out=S2, ws=ws)
        assert torch.equal(o, o2) and torch.equal(S, S2)


# ---------------------------------------------------------------- the Python layer

def test_a_state_out_that_is_not_wanted_is_refused():
    import torch
    import byte_level_lm_amd as B
    x, off = torch.zeros(4, 1, 8), torch.tensor([0, 4])
    with pytest.raises(ValueError, match="state_out needs want_state"):
        B.gated_delta(x, x, x, x[:, :, 0], x[:, :, 0], off, want_state=False, state_out=torch.zeros(1, 1, 8, 8))


def test_the_current_stream_without_the_raw_call(monkeypatch):
    """A torch that lacks the raw handle's call: the binding takes the public one."""
    import importlib.util
    import types
    import torch
    from byte_level_lm_amd import ops
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1234))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    spec = importlib.util.spec_from_file_location("byte_level_lm_amd._ops_again", ops.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._stream() == 1234


@pytest.mark.gpu
def test_calls_go_to_the_current_stream(B):
    import torch
    from byte_level_lm_amd import ops
    assert ops._stream() == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert ops._stream() == side.cuda_stream != 0
    assert ops._stream() == torch.cuda.current_stream().cuda_stream
