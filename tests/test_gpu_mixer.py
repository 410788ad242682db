"""GPU parity of the mixer block's operators against the 64-bit oracle.

Tolerances, from the roundings each result goes through:
  * integer codes and sums are exact;
  * an output rounded to bf16 (8 significant bits) is within 2^-8 of its value in each element;
    fp32 outputs of a norm or a product take at most 8 fp32 roundings
    (2^-21 in all) beside a tree sum whose error stays under 2^-20;
  * the gated delta rule: states are kept to 24 bits through sums of at most
    128 + 64 products (192 * 2^-24 < 1.2e-5 in the norm of a head); outputs add
    their own rounding and at most one operand rounded to 8 bits, whose errors lie
    evenly within 2^-8 of each element: below 2^-9 each in the norm of a row.
"""
import numpy as np
import pytest

import oracle
from synthdata import bf16_round
from tests.helpers import to_dev, to_np, row_rel_err, say

pytestmark = pytest.mark.gpu

F32_TOL = 2.0 ** -20 + 2.0 ** -21
BF16_TOL = 2.0 ** -8 * 1.01
STATE_TOL = 1.2e-5
O_TOL = 2.0 ** -8 * 1.02


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rows(rng, shape, dtype, scale=1.0):
    x = (scale * rng.standard_normal(shape)).astype(np.float32)
    return bf16_round(x) if dtype == "bf16" else x


# ---------------------------------------------------------------- norms and 8-bit rows

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 64), (129, 512), (37, 520), (300, 768), (5, 1536), (9, 4096), (2, 16392),
                                    (2, 40000)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_and_q8(B, dtype, rows, d, residual):
    rng = np.random.default_rng(rows * 7 + d)
    say("rmsnorm", dtype, rows, d, residual)
    x, w = _rows(rng, (rows, d), dtype), bf16_round(1 + 0.2 * rng.standard_normal(d).astype(np.float32))
    r = _rows(rng, (rows, d), dtype, 2.0) if residual else None
    dt = _dt(dtype)
    dx, dw, dr = to_dev(x, dt), to_dev(w, dt), None if r is None else to_dev(r, dt)
    y_o, s_o = oracle.rmsnorm(x, w, 1e-6, r)
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    y, res = B.rmsnorm(dx, dw, eps=1e-6, residual=dr)
    assert np.all(np.abs(to_np(y) - y_o) <= tol * np.abs(y_o) + 1e-30)
    q, scale, res8 = B.rmsnorm_q8(dx, dw, eps=1e-6, residual=dr)
    q_o, scale_o, _ = oracle.rmsnorm_q8(x, w, 1e-6, r)
    assert np.array_equal(to_np(q), q_o)
    np.testing.assert_allclose(to_np(scale), scale_o, rtol=F32_TOL)
    if residual:
        # one fp32 addition, then one rounding to the type: bit for bit
        want = (x + r) if dtype == "f32" else bf16_round(x + r)
        assert np.array_equal(to_np(res), want) and np.array_equal(to_np(res8), want)
    else:
        assert res is None and res8 is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (257, 512), (3, 1544), (2, 20000)])
def test_quant_rows(B, dtype, rows, d):
    rng = np.random.default_rng(d)
    x = _rows(rng, (rows, d), dtype, 3.0)
    q, scale = B.quant_rows_q8(to_dev(x, _dt(dtype)))
    q_o, step = oracle.quant_rows_q8(x)
    assert np.array_equal(to_np(q), q_o)
    np.testing.assert_allclose(to_np(scale), step, rtol=F32_TOL)


def test_norm_special_rows(B):
    """Zero rows, rows too small to divide by, NaN and infinity in one row
    (and only there), values whose ties go to even."""
    x = np.zeros((6, 64), np.float32)
    x[1, 5] = 1e-35
    x[2] = 1.0; x[2, 9] = np.nan
    x[3] = 1.0; x[3, 60] = np.inf
    x[4, :5] = [127.0, 0.5, 1.5, 2.5, -2.5]
    x[5] = np.linspace(-1, 1, 64)
    w = np.ones(64, np.float32)
    q, scale = B.quant_rows_q8(to_dev(x))
    q, scale = to_np(q), to_np(scale)
    assert not q[0].any() and scale[0] == 0 and not q[1].any() and scale[1] == 0
    assert not np.isfinite(scale[2]) and not np.isfinite(scale[3])
    assert list(q[4, :5]) == [127, 0, 2, 2, -2] and scale[4] == 1.0
    qn, sn, _ = B.rmsnorm_q8(to_dev(x), to_dev(w))
    qn, sn = to_np(qn), to_np(sn)
    assert not qn[0].any() and sn[0] == 0 and np.isnan(sn[2]) and np.isnan(sn[3])
    assert np.array_equal(qn[[4, 5]], q[[4, 5]])
    y, _ = B.rmsnorm(to_dev(x), to_dev(w))
    y = to_np(y)
    assert np.all(y[0] == 0) and np.all(np.isnan(y[2])) and np.all(np.isfinite(y[[0, 1, 4, 5]]))


def test_norm_in_place_no_rows_and_another_stream(B):
    import torch
    rng = np.random.default_rng(3)
    x, r, w = (_rows(rng, s, "bf16") for s in ((70, 512), (70, 512), (512,)))
    dx, dr, dw = (to_dev(a, torch.bfloat16) for a in (x, r, w))
    y0, s0 = B.rmsnorm(dx, dw, residual=dr)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        y1, s1 = B.rmsnorm(dx, dw, residual=dr, residual_out=dr, y_out=dx)
    torch.cuda.current_stream().wait_stream(stream)
    assert y1.data_ptr() == dx.data_ptr() and s1.data_ptr() == dr.data_ptr()
    assert torch.equal(y0, y1) and torch.equal(s0, s1)
    y, res = B.rmsnorm(dx[:0], dw)
    q, scale, _ = B.rmsnorm_q8(dx[:0], dw)
    assert y.shape == (0, 512) and res is None and q.shape == (0, 512) and scale.shape == (0,)


# ---------------------------------------------------------------- 8-bit product

LIN = [(1, 1, 16), (1, 512, 512), (3, 17, 48), (16, 1536, 512), (17, 96, 1040), (33, 130, 80), (64, 64, 64),
       (100, 777, 4096), (129, 257, 768), (300, 40, 131056), (257, 512, 192), (1000, 1551, 336), (2, 8192, 128),
       (513, 1024, 2048),
       # tiles of 128 x 128 and of 256 x 256, several of those a workgroup, K shorter than a step or ending inside one
       (2048, 2100, 80), (4000, 2200, 144), (9000, 2200, 48), (4100, 2060, 336), (6200, 2060, 336)]


@pytest.mark.parametrize("m,n,k", LIN)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_i8(B, m, n, k, out):
    rng = np.random.default_rng(m + n + k)
    say("linear_i8", m, n, k, out)
    xq, wq = rng.integers(-128, 128, (m, k), dtype=np.int8), rng.integers(-128, 128, (n, k), dtype=np.int8)
    sx, sw = (rng.random(m) + 0.1).astype(np.float32), (rng.random(n) + 0.1).astype(np.float32)
    bias = (1e4 * rng.standard_normal(n)).astype(np.float32) if m % 2 else None
    acc = np.rint(xq.astype(np.float64) @ wq.T.astype(np.float64))  # whole numbers below 2^53: exact
    y_o = acc * sx.astype(np.float64)[:, None] * sw + (0 if bias is None else bias)
    y = B.linear_i8(to_dev(xq), to_dev(sx), to_dev(wq), to_dev(sw), bias=None if bias is None else to_dev(bias),
                    out_dtype=_dt(out))
    # fp32 steps: int to float, two products, one sum, each 2^-24 of its size
    slack = 2.0 ** -22 * (np.abs(acc) * sx[:, None] * sw + (0 if bias is None else np.abs(bias)))
    if out == "bf16":
        slack = slack * 1.01 + BF16_TOL * np.abs(y_o)
    assert np.all(np.abs(to_np(y) - y_o) <= slack)


def test_linear_i8_extreme_sums_rows_apart_and_edges(B):
    """The largest sum that fits; a row's NaN scale stays in its row; the bytes
    behind the last row and column are not written."""
    import torch
    k = 131056
    xq, wq = np.full((2, k), -128, np.int8), np.full((3, k), -128, np.int8)
    y = B.linear_i8(to_dev(xq), to_dev(np.ones(2, np.float32)), to_dev(wq), to_dev(np.ones(3, np.float32)),
                    out_dtype=torch.float32)
    assert np.all(to_np(y) == np.float32(128.0 * 128.0 * k))
    for m, n in [(5, 7), (70, 131), (300, 259)]:
        buf = torch.full((m * n + 64,), 7.0, device="cuda")
        sx = np.ones(m, np.float32); sx[2] = np.nan
        rng = np.random.default_rng(m)
        a, b = rng.integers(-9, 10, (m, 64), dtype=np.int8), rng.integers(-9, 10, (n, 64), dtype=np.int8)
        y = B.linear_i8(to_dev(a), to_dev(sx), to_dev(b), to_dev(np.ones(n, np.float32)),
                        y_out=buf[:m * n].view(m, n))
        want = oracle.linear_i8(a, np.ones(m), b, np.ones(n))
        got = to_np(y)
        assert np.all(np.isnan(got[2])) and np.array_equal(np.delete(got, 2, 0), np.delete(want, 2, 0))
        assert torch.all(buf[m * n:] == 7.0)
    assert B.linear_i8(to_dev(xq[:0]), to_dev(np.ones(0, np.float32)), to_dev(wq), to_dev(np.ones(3, np.float32))).shape == (0, 3)


# ---------------------------------------------------------------- gated delta rule

def _delta_inputs(rng, lengths, hk, hv, dk, dv, spread=0.3):
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(off[-1])
    q, k = (bf16_round(rng.standard_normal((n, hk, dk)).astype(np.float32)) for _ in range(2))
    v = bf16_round(rng.standard_normal((n, hv, dv)).astype(np.float32))
    g = (-spread * rng.random((n, hv)) ** 3).astype(np.float32)
    beta = rng.random((n, hv)).astype(np.float32)
    return off, q, k, v, g, beta


def _strided(q, k, v):
    """q, k, v as column slices of one row-major array, as a projection gives them."""
    import torch
    n = q.shape[0]
    row = np.concatenate([a.reshape(n, -1) for a in (q, k, v)], axis=1)
    row = to_dev(row, torch.bfloat16)
    cut = np.cumsum([0, q[0].size, k[0].size, v[0].size])
    return [row[:, cut[i]:cut[i + 1]].unflatten(1, a.shape[1:]) for i, a in enumerate((q, k, v))]


def _check_delta(o, S, o_o, S_o):
    S = to_np(S).reshape(S_o.shape[0] * S_o.shape[1], -1)
    assert row_rel_err(S, S_o.reshape(S.shape)) <= STATE_TOL
    # a token's output can cancel: its error is measured against the head's typical row
    o = to_np(o).astype(np.float64)
    rms = np.sqrt(np.mean(o_o ** 2, axis=(0, 2), keepdims=True)) if o_o.size else 1.0
    size = np.maximum(np.linalg.norm(o_o, axis=2, keepdims=True), rms * np.sqrt(o_o.shape[2]))
    assert o_o.size == 0 or np.max(np.linalg.norm(o - o_o, axis=2, keepdims=True) / np.maximum(size, 1e-30)) <= O_TOL


DELTA = [
    ([1], 1, 1, 8, 8), ([5], 1, 1, 16, 16), ([63, 64, 65], 1, 2, 64, 64), ([0, 3, 0, 130, 1], 2, 2, 128, 128),
    ([200], 2, 6, 32, 40), ([77, 128], 3, 3, 40, 24), ([300, 17], 1, 1, 128, 256), ([129], 2, 2, 96, 72),
    ([7] * 40, 1, 4, 64, 32), ([520], 1, 1, 72, 136), ([1000, 0, 10], 1, 1, 64, 128),
    # enough heads and columns that a workgroup takes 64 columns; the others split a head's columns in sixteens
    ([70, 0, 9, 64] * 8, 2, 8, 128, 72), ([65, 3] * 20, 1, 8, 24, 40), ([33, 66] * 16, 8, 8, 128, 64),
    ([80, 1] * 16, 1, 8, 64, 128),
    # long sequences of few heads, in segments
    ([1600], 2, 2, 128, 128), ([1700], 1, 4, 64, 40), ([3000, 0, 100], 1, 1, 40, 24), ([1024], 1, 1, 128, 8),
    ([64 * 21], 1, 2, 72, 136), ([1153, 1200], 1, 1, 8, 64),
    # few tokens a sequence on average, one of them long
    ([1, 0, 2] * 10 + [90], 2, 4, 64, 40), ([3, 5], 1, 2, 104, 136),
]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", DELTA)
@pytest.mark.parametrize("state,unit", [(False, True), (True, True), (True, False)])
def test_gated_delta(B, lengths, hk, hv, dk, dv, state, unit):
    rng = np.random.default_rng(sum(lengths) + dk + dv)
    say("gated_delta", lengths[:5], hk, hv, dk, dv, state, unit)
    off, q, k, v, g, beta = _delta_inputs(rng, lengths, hk, hv, dk, dv)
    if not unit:
        q, k = bf16_round(q / np.sqrt(dk)), bf16_round(k / np.linalg.norm(k, axis=2, keepdims=True))
    S0 = rng.standard_normal((len(lengths), hv, dk, dv)).astype(np.float32) if state else None
    scale = dk ** -0.5
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=scale, unit_qk=unit, state=S0)
    dS = to_dev(S0) if state else None
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off), state_in=dS, state_out=dS,
                         unit_qk=unit)
    assert not state or S.data_ptr() == dS.data_ptr()
    _check_delta(o, S, o_o, S_o)


@pytest.mark.parametrize("length", [40, 200])
def test_gated_delta_gates_at_their_ends(B, length):
    """Decays of 0 (forget), 1, and e^-100; write strengths 0, 1 and 2; a state
    is passed on without decay through beta = 0."""
    rng = np.random.default_rng(length)
    off, q, k, v, g, beta = _delta_inputs(rng, [length, length, length], 2, 2, 64, 64)
    g[::7] = -np.inf
    g[3::11] = -100.0
    g[5::13] = 0.0
    beta[::5] = 0.0
    beta[1::9] = 2.0
    a, b = int(off[1]), int(off[2])
    g[a:b] = 0.0; beta[a:b] = 0.0
    S0 = rng.standard_normal((3, 2, 64, 64)).astype(np.float32)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=0.125, unit_qk=True, state=S0)
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off), state_in=to_dev(S0))
    _check_delta(o, S, o_o, S_o)
    assert np.array_equal(to_np(S)[1], S0[1])


def test_gated_delta_nonfinite_stays_in_its_sequence_and_head(B):
    rng = np.random.default_rng(8)
    off, q, k, v, g, beta = _delta_inputs(rng, [100, 90, 130], 2, 2, 64, 64)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=0.125, unit_qk=True)
    v[150, 1, 3] = np.nan  # sequence 1, head 1
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off))
    o, S = to_np(o), to_np(S)
    assert np.isnan(S[1, 1]).any() and np.isnan(o[150:190, 1, 3]).all()
    for s, h in [(0, 0), (0, 1), (1, 0), (2, 0), (2, 1)]:
        assert row_rel_err(S[s, h].reshape(1, -1), S_o[s, h].reshape(1, -1)) <= STATE_TOL
    assert np.isfinite(o[:150]).all() and np.isfinite(o[190:]).all() and np.isfinite(o[150:190, 0]).all()


@pytest.mark.parametrize("nseq", [3, 40])
@pytest.mark.parametrize("what", ["v nan", "v inf", "k nan", "q inf", "state"])
def test_gated_delta_nonfinite_stays_after_its_token_and_in_its_column(B, nseq, what):
    """With few and with many heads: one value that is not finite in sequence 1, head 1, token 70 (or in its state)."""
    rng = np.random.default_rng(16)
    off, q, k, v, g, beta = _delta_inputs(rng, [150] * nseq, 2, 2, 128, 64)
    S0 = rng.standard_normal((nseq, 2, 128, 64)).astype(np.float32)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=128 ** -0.5, unit_qk=True, state=S0)
    at, end = 150 + 70, 300
    lost, gone = np.zeros(o_o.shape, bool), np.zeros(S_o.shape, bool)
    if what[0] == "v":
        v[at, 1, 3] = np.nan if what == "v nan" else np.inf
        lost[at:end, 1, 3] = True
        gone[1, 1, :, 3] = True
    elif what[0] == "k":
        k[at, 1, 5] = np.nan
        lost[at:end, 1] = True
        gone[1, 1] = True
    elif what[0] == "q":
        q[at, 1, 5] = np.inf
        lost[at, 1] = True
    else:
        S0[1, 1, 9, 33] = -np.inf
        lost[150:end, 1, 33] = True
        gone[1, 1, :, 33] = True
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off), state_in=to_dev(S0))
    o, S = to_np(o), to_np(S)
    assert not np.isfinite(o[lost]).any() and not np.isfinite(S[gone]).any()
    assert np.isfinite(o[~lost]).all() and np.isfinite(S[~gone]).all()
    _check_delta(to_dev(np.where(lost, o_o, o).astype(np.float32)), to_dev(np.where(gone, S_o, S).astype(np.float32)), o_o, S_o)


@pytest.mark.parametrize("what", ["v nan", "k inf", "state", "gate"])
def test_gated_delta_nonfinite_in_a_long_sequence(B, what):
    """The same where a sequence of few heads goes in segments: what is lost starts at token 900 of head 1 (or at 0)."""
    rng = np.random.default_rng(17)
    off, q, k, v, g, beta = _delta_inputs(rng, [2000], 1, 2, 64, 48, spread=0.05)
    S0 = rng.standard_normal((1, 2, 64, 48)).astype(np.float32)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=0.125, unit_qk=True, state=S0)
    lost, gone = np.zeros(o_o.shape, bool), np.zeros(S_o.shape, bool)
    if what == "v nan":
        v[900, 1, 3] = np.nan
        lost[900:, 1, 3] = True
        gone[0, 1, :, 3] = True
    elif what == "state":
        S0[0, 1, 9, 33] = np.nan
        lost[:, 1, 33] = True
        gone[0, 1, :, 33] = True
    elif what == "gate":
        g[900, 1] = np.nan
        lost[900:, 1] = True
        gone[0, 1] = True
    else:  # the key's heads share it
        k[900, 0, 5] = np.inf
        lost[900:] = True
        gone[0] = True
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off), state_in=to_dev(S0))
    o, S = to_np(o), to_np(S)
    assert not np.isfinite(o[lost]).any() and not np.isfinite(S[gone]).any()
    assert np.isfinite(o[~lost]).all() and np.isfinite(S[~gone]).all()
    _check_delta(to_dev(np.where(lost, o_o, o).astype(np.float32)), to_dev(np.where(gone, S_o, S).astype(np.float32)), o_o, S_o)


def test_gated_delta_windows_equal_the_whole_and_long_stream(B):
    """A stream in windows with the state carried equals the stream at once, over
    many blocks; no state wanted; no tokens at all."""
    import torch
    rng = np.random.default_rng(9)
    off, q, k, v, g, beta = _delta_inputs(rng, [1500], 1, 2, 128, 128, spread=0.05)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=128 ** -0.5, unit_qk=True)
    dq, dk_, dv_, dg, db = *_strided(q, k, v), to_dev(g), to_dev(beta)
    o, S = B.gated_delta(dq, dk_, dv_, dg, db, to_dev(off))
    _check_delta(o, S, o_o, S_o)
    st, parts = None, []
    for a, b in [(0, 64), (64, 65), (65, 1000), (1000, 1000), (1000, 1500)]:
        cut = to_dev(np.array([0, b - a], np.int64))
        po, st = B.gated_delta(dq[a:b], dk_[a:b], dv_[a:b], dg[a:b], db[a:b], cut, state_in=st)
        parts.append(po)
    _check_delta(torch.cat(parts), st, o_o, S_o)
    o2, none = B.gated_delta(dq, dk_, dv_, dg, db, to_dev(off), want_state=False)
    assert none is None and torch.equal(o, o2)


def test_gated_delta_offsets_outside_the_batch_stay_inside(B):
    """Offsets past the rows are cut at them: nothing outside o or the states is touched."""
    import torch
    rng = np.random.default_rng(10)
    off, q, k, v, g, beta = _delta_inputs(rng, [100, 60], 1, 1, 64, 64)
    buf = torch.full((160 * 64 + 4096,), 5.0, dtype=torch.bfloat16, device="cuda")
    bad = np.array([0, 100, 900], np.int64)
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(bad),
                         o_out=buf[:160 * 64].view(160, 1, 64))
    assert torch.all(buf[160 * 64:] == 5.0)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=0.125, unit_qk=True)
    _check_delta(o, S, o_o, S_o)


@pytest.mark.parametrize("lengths,hv,dk,dv", [([2000], 2, 128, 128), ([1700, 64, 1], 1, 64, 40), ([1024], 1, 8, 8),
                                              ([150] * 40, 8, 128, 64), ([130], 1, 72, 136)])
def test_gated_delta_stays_in_its_workspace(B, lengths, hv, dk, dv):
    """The size that the library names is enough: nothing behind it is written; a smaller one is refused."""
    import torch
    rng = np.random.default_rng(18)
    say("workspace", lengths[:3], hv, dk, dv)
    off, q, k, v, g, beta = _delta_inputs(rng, lengths, hv, hv, dk, dv, spread=0.05)
    size = B.gated_delta_workspace(len(lengths), int(off[-1]), hv, dk, dv)
    buf = torch.full((size + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    S0 = rng.standard_normal((len(lengths), hv, dk, dv)).astype(np.float32)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=dk ** -0.5, unit_qk=True, state=S0)
    args = (*_strided(q, k, v), to_dev(g), to_dev(beta), to_dev(off))
    o, S = B.gated_delta(*args, state_in=to_dev(S0), ws=buf[:size])
    _check_delta(o, S, o_o, S_o)
    assert torch.all(buf[size:] == 0x5A)
    with pytest.raises(ValueError):
        B.gated_delta(*args, state_in=to_dev(S0), ws=buf[:size - 4])


@pytest.mark.parametrize("nseq,hk,hv,dk,dv", [(1, 1, 1, 8, 8), (1, 4, 4, 128, 128), (5, 2, 4, 64, 64), (33, 1, 3, 40, 72),
                                              (3, 1, 1, 16, 1024), (130, 2, 2, 128, 32)])
@pytest.mark.parametrize("unit", [True, False])
def test_gated_delta_step(B, nseq, hk, hv, dk, dv, unit):
    import torch
    rng = np.random.default_rng(nseq + dk + dv)
    say("gated_delta_step", nseq, hk, hv, dk, dv, unit)
    off, q, k, v, g, beta = _delta_inputs(rng, [1] * nseq, hk, hv, dk, dv)
    if not unit:
        k = bf16_round(k / np.linalg.norm(k, axis=2, keepdims=True))
    S0 = rng.standard_normal((nseq, hv, dk, dv)).astype(np.float32)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=dk ** -0.5, unit_qk=unit, state=S0)
    dq, dk_, dv_ = _strided(q, k, v)
    o, S = B.gated_delta_step(dq, dk_, dv_, to_dev(g), to_dev(beta), to_dev(S0), unit_qk=unit)
    _check_delta(o, S, o_o, S_o)
    # slots of a pool, in place; two streams without a slot start from zero and keep nothing
    pool = rng.standard_normal((nseq + 3, hv, dk, dv)).astype(np.float32)
    slots = rng.permutation(nseq + 3)[:nseq].astype(np.int32)
    pool[slots] = S0
    slots[0] = -1
    if nseq > 1:
        slots[-1] = nseq + 3
    d = to_dev(pool)
    o, S = B.gated_delta_step(dq, dk_, dv_, to_dev(g), to_dev(beta), d, slots=to_dev(slots), unit_qk=unit)
    S0[slots < 0] = 0
    S0[slots >= nseq + 3] = 0
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=dk ** -0.5, unit_qk=unit, state=S0)
    kept = (slots >= 0) & (slots < nseq + 3)
    want = pool.copy()
    want[slots[kept]] = S_o[kept]
    got = to_np(S)
    rest = np.setdiff1d(np.arange(nseq + 3), slots[kept])
    assert np.array_equal(got[rest], pool[rest])
    _check_delta(o, S, o_o, want)


@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_gated_delta_equal_keys(B, beta):
    """One key for all tokens: the state holds the last values only (strength 1) or reflects (2)."""
    rng = np.random.default_rng(14)
    off, q, k, v, g, b = _delta_inputs(rng, [150], 1, 1, 64, 64)
    k[:] = k[0]
    g[:] = 0.0
    b[:] = beta
    o_o, S_o = oracle.gated_delta(q, k, v, g, b, off, scale=0.125, unit_qk=True)
    o, S = B.gated_delta(*_strided(q, k, v), to_dev(g), to_dev(b), to_dev(off))
    _check_delta(o, S, o_o, S_o)


def test_offsets_past_32_bits(B):
    """Rows, outputs and pool slots whose element numbers pass 2^31 and 2^32."""
    import torch
    rng = np.random.default_rng(15)
    n, d = 1_100_000, 2048
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    last = _rows(rng, (3, d), "bf16")
    x[-3:] = to_dev(last, torch.bfloat16)
    q, scale, _ = B.rmsnorm_q8(x, torch.ones(d, dtype=torch.bfloat16, device="cuda"))
    q_o, _, _ = oracle.rmsnorm_q8(last, np.ones(d, np.float32), 1e-6)
    assert np.array_equal(to_np(q[-3:]), q_o) and not q[0].any()
    del x, q
    m, n, k = 70_000, 32_768, 16
    a, b = rng.integers(-128, 128, (m, k), dtype=np.int8), rng.integers(-128, 128, (n, k), dtype=np.int8)
    y = B.linear_i8(to_dev(a), to_dev(np.ones(m, np.float32)), to_dev(b), to_dev(np.ones(n, np.float32)),
                    out_dtype=torch.float32)
    assert np.array_equal(to_np(y[-300:, -300:]), oracle.linear_i8(a[-300:], np.ones(300), b[-300:], np.ones(300)))
    del y
    slots, hv, dk = 70_000, 4, 128
    pool = torch.empty(slots, hv, dk, dk, device="cuda")
    off, q, k, v, g, beta = _delta_inputs(rng, [1] * 3, 2, hv, dk, dk)
    at = np.array([slots - 1, 0, 33_000], np.int32)
    S0 = rng.standard_normal((3, hv, dk, dk)).astype(np.float32)
    pool[torch.from_numpy(at.astype(np.int64)).cuda()] = to_dev(S0)
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=dk ** -0.5, unit_qk=True, state=S0)
    o, _ = B.gated_delta_step(*_strided(q, k, v), to_dev(g), to_dev(beta), pool, slots=to_dev(at))
    _check_delta(o, pool[torch.from_numpy(at.astype(np.int64)).cuda()], o_o, S_o)
    del pool
    # one long sequence before a short one: the short one's rows lie past 2^31 elements of v and o
    long, short, hv, dv = 700_000, 100, 32, 128
    off, q, k, v, g, beta = _delta_inputs(rng, [short], 1, hv, 8, dv)
    dv_ = torch.zeros(long + short, hv, dv, dtype=torch.bfloat16, device="cuda")
    dq, dk_ = (torch.zeros(long + short, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg, db = (torch.zeros(long + short, hv, device="cuda") for _ in range(2))
    for t, a in ((dv_, v), (dq, q), (dk_, k), (dg, g), (db, beta)):
        t[long:] = to_dev(a, t.dtype)
    o, S = B.gated_delta(dq, dk_, dv_, dg, db, to_dev(np.array([0, long, long + short])))
    o_o, S_o = oracle.gated_delta(q, k, v, g, beta, off, scale=8 ** -0.5, unit_qk=True)
    _check_delta(o[long:], S[1:], o_o, S_o)
    assert not S[0].any() and not o[:64].any()


def test_operators_inside_a_captured_graph(B):
    """One block's calls captured once and replayed on new inputs, eager work in between."""
    import torch
    rng = np.random.default_rng(12)
    d, hk, dk, n = 128, 2, 64, 150
    w8, ws = B.quant_rows_q8(to_dev(rng.standard_normal((3 * d, d)).astype(np.float32)))
    nw = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    x, r = (torch.zeros(n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g, beta = -0.1 * torch.rand(n, hk, device="cuda"), torch.rand(n, hk, device="cuda")
    off = to_dev(np.array([0, 100, 150], np.int64))

    def block():
        q8, s8, res = B.rmsnorm_q8(x, nw, residual=r)
        qkv = B.linear_i8(q8, s8, w8, ws)
        q, k, v = (qkv[:, i * d:(i + 1) * d].unflatten(1, (hk, dk)) for i in range(3))
        o, S = B.gated_delta(q, k, v, g, beta, off)
        o1, S1 = B.gated_delta_step(q[:2], k[:2], v[:2], g[:2], beta[:2], S, state_out=torch.empty_like(S))
        return res, o, S, o1, S1

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for i in range(4):
        torch.manual_seed(i)
        x.copy_(torch.randn(n, d)); r.copy_(torch.randn(n, d))
        want = [t.clone() for t in block()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
