"""Python binding of the chunk-layer C ABI (same names as include/bllm.h).

Argument marshalling only: each function checks shapes and dtypes, allocates
outputs/workspaces with torch when the caller does not pass them, and calls
the HIP library on torch's current stream.  Every step of the computation
runs in the library's kernels.  Nothing here synchronises: data-dependent
results (counts, status words) stay on the device until the caller reads them.
"""
from __future__ import annotations

import torch

from . import _lib as L


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return L.F32
    if t.dtype == torch.bfloat16:
        return L.BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on the GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


# the raw handle of the current stream without building a Stream object; not a public name of torch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _ws(nbytes: int, ws, device):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return ws
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _nbytes(t):
    return t.numel() * t.element_size()


# ------------------------------------------------------------------ sizes

def route_workspace(total: int) -> int:
    return int(L.lib().bllm_route_workspace(total))


def compact_workspace(total: int) -> int:
    return int(L.lib().bllm_compact_workspace(total))


def dechunk_workspace(d: int) -> int:
    return int(L.lib().bllm_dechunk_workspace(d))


def coding_rate_workspace(nseq: int, T: int, d: int) -> int:
    return int(L.lib().bllm_coding_rate_workspace(nseq, T, d))


def upsample_workspace(nseq: int, T: int, K: int, d_global: int, d_local: int, nbins: int) -> int:
    return int(L.lib().bllm_upsample_workspace(nseq, T, K, d_global, d_local, nbins))


# ------------------------------------------------------------------ ops

def route(q, k, offsets, *, threshold: float = 0.5, quantile=None, p_out=None, b_out=None,
          tau_out=None, status=None, ws=None):
    """H-Net boundary scores p, mask b and threshold tau (device tensors).
    `status` (int32 [1], device, optional) receives BLLM_S_INCOMPLETE if the
    quantile's bounded device-side wait gave up."""
    _dev(q, k, offsets)
    total, d = q.shape
    if k.shape != q.shape or k.dtype != q.dtype or offsets.dtype != torch.int64:
        raise ValueError("q and k must match; offsets must be int64")
    dev = q.device
    p_out = torch.empty(total, dtype=torch.float32, device=dev) if p_out is None else p_out
    b_out = torch.empty(total, dtype=torch.uint8, device=dev) if b_out is None else b_out
    tau_out = torch.empty(1, dtype=torch.float32, device=dev) if tau_out is None else tau_out
    quant = -1.0 if quantile is None else float(quantile)
    w = _ws(route_workspace(total), ws, dev) if quantile is not None else ws
    rc = L.lib().bllm_route(q.data_ptr(), k.data_ptr(), _dt(q), d, offsets.data_ptr(),
                            offsets.numel() - 1, total, float(threshold), quant, p_out.data_ptr(),
                            b_out.data_ptr(), tau_out.data_ptr(), _ptr(status), _ptr(w),
                            0 if w is None else _nbytes(w), _stream())
    L.check("bllm_route", rc)
    return p_out, b_out, tau_out


def route_fused(h, Wq, Wk, offsets, *, threshold: float = 0.5, quantile=None, p_out=None, b_out=None,
                tau_out=None, status=None, ws=None):
    """bllm_route with q = h Wq and k = h Wk formed inside the kernel (bf16 h, Wq, Wk)."""
    _dev(h, Wq, Wk, offsets)
    total, d = h.shape
    dev = h.device
    p_out = torch.empty(total, dtype=torch.float32, device=dev) if p_out is None else p_out
    b_out = torch.empty(total, dtype=torch.uint8, device=dev) if b_out is None else b_out
    tau_out = torch.empty(1, dtype=torch.float32, device=dev) if tau_out is None else tau_out
    w = _ws(route_workspace(total), ws, dev) if quantile is not None else ws
    rc = L.lib().bllm_route_fused(h.data_ptr(), Wq.data_ptr(), Wk.data_ptr(), _dt(h), d, offsets.data_ptr(),
                                  offsets.numel() - 1, total, float(threshold),
                                  -1.0 if quantile is None else float(quantile), p_out.data_ptr(),
                                  b_out.data_ptr(), tau_out.data_ptr(), _ptr(status), _ptr(w),
                                  0 if w is None else _nbytes(w), _stream())
    L.check("bllm_route_fused", rc)
    return p_out, b_out, tau_out


def compact(mask, offsets, *, rows=None, p=None, capacity=None, idx_out=None,
            chunk_offsets_out=None, rows_out=None, P_out=None, status=None, ws=None):
    """Keep set mask positions: returns (idx, chunk_offsets, rows_out, P_out, status).
    Outputs have `capacity` rows; the true count is chunk_offsets[-1] (on device)."""
    _dev(mask, offsets, rows, p)
    total = mask.numel()
    nseq = offsets.numel() - 1
    dev = mask.device
    cap = total if capacity is None else int(capacity)
    idx_out = torch.empty(max(cap, 1), dtype=torch.int32, device=dev) if idx_out is None else idx_out
    chunk_offsets_out = (torch.empty(nseq + 1, dtype=torch.int64, device=dev)
                         if chunk_offsets_out is None else chunk_offsets_out)
    d = 0
    dt = L.F32
    if rows is not None:
        d = rows.shape[1]
        dt = _dt(rows)
        if rows_out is None:
            rows_out = torch.empty((max(cap, 1), d), dtype=rows.dtype, device=dev)
    if p is not None and P_out is None:
        P_out = torch.empty(max(cap, 1), dtype=torch.float32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    w = _ws(compact_workspace(total), ws, dev)
    rc = L.lib().bllm_compact(mask.data_ptr(), _ptr(p), _ptr(rows), dt, d, offsets.data_ptr(), nseq,
                              total, cap, idx_out.data_ptr(), chunk_offsets_out.data_ptr(),
                              _ptr(rows_out), _ptr(P_out), status.data_ptr(), w.data_ptr(),
                              _nbytes(w), _stream())
    L.check("bllm_compact", rc)
    return idx_out, chunk_offsets_out, rows_out, P_out, status


def compact_noalloc(mask, offsets, *, rows=None, p=None, capacity=None, idx_out=None,
                    chunk_offsets_out=None, rows_out=None, P_out=None, status=None):
    """bllm_compact on the library's own scratch array (no workspace; at most
    2^27 positions).  Outputs must be passed in by a caller that cannot
    allocate; any left as None are allocated here for convenience."""
    _dev(mask, offsets, rows, p)
    total = mask.numel()
    nseq = offsets.numel() - 1
    dev = mask.device
    cap = total if capacity is None else int(capacity)
    idx_out = torch.empty(max(cap, 1), dtype=torch.int32, device=dev) if idx_out is None else idx_out
    chunk_offsets_out = (torch.empty(nseq + 1, dtype=torch.int64, device=dev)
                         if chunk_offsets_out is None else chunk_offsets_out)
    d = 0
    dt = L.F32
    if rows is not None:
        d = rows.shape[1]
        dt = _dt(rows)
        if rows_out is None:
            rows_out = torch.empty((max(cap, 1), d), dtype=rows.dtype, device=dev)
    if p is not None and P_out is None:
        P_out = torch.empty(max(cap, 1), dtype=torch.float32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    rc = L.lib().bllm_compact_noalloc(mask.data_ptr(), _ptr(p), _ptr(rows), dt, d, offsets.data_ptr(), nseq,
                                      total, cap, idx_out.data_ptr(), chunk_offsets_out.data_ptr(),
                                      _ptr(rows_out), _ptr(P_out), status.data_ptr(), _stream())
    L.check("bllm_compact_noalloc", rc)
    return idx_out, chunk_offsets_out, rows_out, P_out, status


def dechunk_ema(z, P, idx, chunk_offsets, offsets, total: int, *, out=None, ws=None,
                max_chunks=None):
    """EMA over chunks expanded back to `total` byte rows."""
    _dev(z, P, idx, chunk_offsets, offsets)
    d = z.shape[1]
    dev = z.device
    out = torch.empty((total, d), dtype=z.dtype, device=dev) if out is None else out
    w = _ws(dechunk_workspace(d), ws, dev)
    mc = z.shape[0] if max_chunks is None else int(max_chunks)
    rc = L.lib().bllm_dechunk_ema(z.data_ptr(), P.data_ptr(), _dt(z), d, idx.data_ptr(),
                                  chunk_offsets.data_ptr(), offsets.data_ptr(), offsets.numel() - 1,
                                  int(total), mc, out.data_ptr(), w.data_ptr(), _nbytes(w),
                                  _stream())
    L.check("bllm_dechunk_ema", rc)
    return out


def dechunk_ema_backward_workspace(d: int, max_chunks: int) -> int:
    return int(L.lib().bllm_dechunk_ema_backward_workspace(d, max_chunks))


def dechunk_ema_backward(z, P, dout, idx, chunk_offsets, offsets, *, dz_out=None, dP_out=None, ws=None,
                         max_chunks=None):
    """Gradients (dz, dP) of sum(dout * dechunk_ema(z, P, ...)) with respect to z and P."""
    _dev(z, P, dout, idx, chunk_offsets, offsets)
    d = z.shape[1]
    dev = z.device
    mc = z.shape[0] if max_chunks is None else int(max_chunks)
    dz_out = torch.empty((mc, d), dtype=z.dtype, device=dev) if dz_out is None else dz_out
    dP_out = torch.empty(mc, dtype=torch.float32, device=dev) if dP_out is None else dP_out
    w = _ws(dechunk_ema_backward_workspace(d, mc), ws, dev)
    rc = L.lib().bllm_dechunk_ema_backward(z.data_ptr(), P.data_ptr(), dout.data_ptr(), _dt(z), d,
                                           idx.data_ptr(), chunk_offsets.data_ptr(), offsets.data_ptr(),
                                           offsets.numel() - 1, dout.shape[0], mc, dz_out.data_ptr(),
                                           dP_out.data_ptr(), w.data_ptr(), _nbytes(w), _stream())
    L.check("bllm_dechunk_ema_backward", rc)
    return dz_out, dP_out


def coding_rate(h, eps2: float, *, dR_out=None, status=None, ws=None):
    """Delta R_t for h [nseq, T, d]; returns (dR fp32 [nseq, T], status)."""
    _dev(h)
    nseq, T, d = h.shape
    dev = h.device
    dR_out = torch.empty((nseq, T), dtype=torch.float32, device=dev) if dR_out is None else dR_out
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    w = _ws(coding_rate_workspace(nseq, T, d), ws, dev)
    rc = L.lib().bllm_coding_rate(h.data_ptr(), _dt(h), nseq, T, d, float(eps2), dR_out.data_ptr(),
                                  status.data_ptr(), w.data_ptr(), _nbytes(w), _stream())
    L.check("bllm_coding_rate", rc)
    return dR_out, status


def coding_rate_split(h, eps2: float, stream2, fork_event, join_event, *, dR_out=None, status=None, ws=None):
    """coding_rate with the batch's second half on `stream2` (a torch.cuda.Stream),
    forked and joined with the caller's two torch.cuda.Event objects."""
    _dev(h)
    nseq, T, d = h.shape
    dev = h.device
    dR_out = torch.empty((nseq, T), dtype=torch.float32, device=dev) if dR_out is None else dR_out
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    w = _ws(coding_rate_workspace(nseq, T, d), ws, dev)
    for ev in (fork_event, join_event):
        if not ev.cuda_event:  # torch creates the event at its first record
            ev.record()
    rc = L.lib().bllm_coding_rate_split(h.data_ptr(), _dt(h), nseq, T, d, float(eps2), dR_out.data_ptr(),
                                        status.data_ptr(), w.data_ptr(), _nbytes(w), _stream(),
                                        stream2.cuda_stream, fork_event.cuda_event, join_event.cuda_event)
    L.check("bllm_coding_rate_split", rc)
    return dR_out, status


def coding_rate_stream(h, eps2: float, state_in=None, *, state_out=None, want_state=True, dR_out=None,
                       status=None, ws=None):
    """Delta R_t of one window h [nseq, W, d] of a stream, given the carried
    prefix matrix state_in (fp32 [nseq, d, d]; None at the stream's start).
    Returns (dR fp32 [nseq, W], state_out fp32 [nseq, d, d] or None, status);
    state_out may be state_in itself (updated in place); want_state=False
    skips the next carry."""
    _dev(h)
    nseq, W, d = h.shape
    dev = h.device
    dR_out = torch.empty((nseq, W), dtype=torch.float32, device=dev) if dR_out is None else dR_out
    if not want_state:
        state_out = None
    elif state_out is None:
        state_out = torch.empty((nseq, d, d), dtype=torch.float32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    w = _ws(coding_rate_workspace(nseq, W, d), ws, dev)
    rc = L.lib().bllm_coding_rate_stream(h.data_ptr(), _dt(h), nseq, W, d, float(eps2), _ptr(state_in),
                                         _ptr(state_out), dR_out.data_ptr(), status.data_ptr(),
                                         w.data_ptr(), _nbytes(w), _stream())
    L.check("bllm_coding_rate_stream", rc)
    return dR_out, state_out, status


def topk_select(score, K: int, *, idx_out=None, mask_out=None, status=None, want_mask=True):
    """BOS + Top-(K-1) positions per sequence in time order: (idx int32, mask uint8, status)."""
    _dev(score)
    nseq, T = score.shape
    dev = score.device
    idx_out = torch.empty((nseq, K), dtype=torch.int32, device=dev) if idx_out is None else idx_out
    if want_mask and mask_out is None:
        mask_out = torch.empty((nseq, T), dtype=torch.uint8, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    rc = L.lib().bllm_topk_select(score.data_ptr(), nseq, T, int(K), idx_out.data_ptr(),
                                  _ptr(mask_out), status.data_ptr(), _stream())
    L.check("bllm_topk_select", rc)
    return idx_out, mask_out, status


def gather_topk(h, idx, *, z_out=None):
    """z [nseq, K, d] = the rows of h [nseq, T, d] at the positions idx [nseq, K] (int32)."""
    _dev(h, idx)
    nseq, T, d = h.shape
    K = idx.shape[1]
    if idx.dtype != torch.int32 or idx.shape[0] != nseq:
        raise ValueError("idx must be int32 [nseq, K]")
    z_out = torch.empty((nseq, K, d), dtype=h.dtype, device=h.device) if z_out is None else z_out
    rc = L.lib().bllm_gather_topk(h.data_ptr(), _dt(h), nseq, T, d, K, idx.data_ptr(), z_out.data_ptr(),
                                  _stream())
    L.check("bllm_gather_topk", rc)
    return z_out


def topk_select_window(score, K: int, first: bool, *, idx_out=None, mask_out=None, status=None, want_mask=True):
    """Local Top-K of one window [nseq, W] of a stream: the first window as
    ``topk_select`` (BOS + K-1), later windows their K largest scores."""
    _dev(score)
    nseq, W = score.shape
    dev = score.device
    idx_out = torch.empty((nseq, K), dtype=torch.int32, device=dev) if idx_out is None else idx_out
    if want_mask and mask_out is None:
        mask_out = torch.empty((nseq, W), dtype=torch.uint8, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    rc = L.lib().bllm_topk_select_window(score.data_ptr(), nseq, W, int(K), 1 if first else 0, idx_out.data_ptr(),
                                         _ptr(mask_out), status.data_ptr(), _stream())
    L.check("bllm_topk_select_window", rc)
    return idx_out, mask_out, status


def upsample_plan(idx, T: int, nbins: int, *, ws=None, d_global: int = 8, d_local: int = 8):
    """The upsample's work items from the chunk starts idx int32 [nseq, K] into a
    workspace (returned; pass it to ``upsample_apply``)."""
    _dev(idx)
    nseq, K = idx.shape
    w = _ws(upsample_workspace(nseq, T, K, d_global, d_local, nbins), ws, idx.device)
    rc = L.lib().bllm_upsample_plan(idx.data_ptr(), nseq, int(T), K, int(nbins), w.data_ptr(), _nbytes(w),
                                    _stream())
    L.check("bllm_upsample_plan", rc)
    return w


def upsample_apply(g, W, h, nbins: int, ws, *, s_out=None):
    """s_t = h_t + g_{c(t)} W_{bin(t)} from a plan made by ``upsample_plan`` in ws."""
    _dev(g, W, h, ws)
    nseq, K, dg = g.shape
    T, dl = h.shape[1], h.shape[2]
    s_out = torch.empty_like(h) if s_out is None else s_out
    rc = L.lib().bllm_upsample_apply(g.data_ptr(), W.data_ptr(), h.data_ptr(), _dt(h), nseq, T, K, dg, dl,
                                     int(nbins), s_out.data_ptr(), ws.data_ptr(), _nbytes(ws), _stream())
    L.check("bllm_upsample_apply", rc)
    return s_out


def upsample_bins(g, W, idx, h, nbins: int, *, s_out=None, ws=None):
    """s_t = h_t + g_{c(t)} W_{bin(t)}; g [nseq,K,dg], W [nbins,dg,dl], idx int32 [nseq,K], h [nseq,T,dl]."""
    _dev(g, W, idx, h)
    nseq, K, dg = g.shape
    T, dl = h.shape[1], h.shape[2]
    dev = h.device
    s_out = torch.empty_like(h) if s_out is None else s_out
    w = _ws(upsample_workspace(nseq, T, K, dg, dl, nbins), ws, dev)
    rc = L.lib().bllm_upsample_bins(g.data_ptr(), W.data_ptr(), idx.data_ptr(), h.data_ptr(), _dt(h),
                                    nseq, T, K, dg, dl, int(nbins), s_out.data_ptr(), w.data_ptr(),
                                    _nbytes(w), _stream())
    L.check("bllm_upsample_bins", rc)
    return s_out


# ------------------------------------------------------------------ mixer block in serving
# A step of one byte makes a dozen of these calls, each a few microseconds on
# the GPU: checks are plain comparisons, and outputs that the caller passes are
# not allocated.

def gated_delta_workspace(nseq: int, total: int, hv: int, dk: int, dv: int) -> int:
    return int(L.lib().bllm_gated_delta_workspace(nseq, total, hv, dk, dv))


def _is(name, t, shape, dtype):
    """t is a dense GPU tensor of this shape and dtype."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        _dev(t)


def _out(name, t, shape, dtype, like):
    """The caller's output, or a new one on the device of ``like``."""
    if t is None:
        if like.shape == shape:  # half the time of building the shape again
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)
    _is(name, t, shape, dtype)
    return t


def _norm_args(x, w, residual, residual_out):
    _dev(x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    _is("w", w, x.shape[1:], x.dtype)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return None
    _is("residual", residual, x.shape, x.dtype)
    return _out("residual_out", residual_out, x.shape, x.dtype, x)


def rmsnorm(x, w, *, eps: float = 1e-6, residual=None, y_out=None, residual_out=None):
    """RMS norm of the rows of x [rows, d] (plus residual), weighted by w [d]:
    returns (y, x + residual), the second None without a residual."""
    residual_out = _norm_args(x, w, residual, residual_out)
    rows, d = x.shape
    y_out = _out("y_out", y_out, x.shape, x.dtype, x)
    rc = L.lib().bllm_rmsnorm(x.data_ptr(), _ptr(residual), w.data_ptr(), _dt(x), rows, d, eps, _ptr(residual_out),
                              y_out.data_ptr(), _stream())
    L.check("bllm_rmsnorm", rc)
    return y_out, residual_out


def rmsnorm_q8(x, w, *, eps: float = 1e-6, residual=None, q_out=None, scale_out=None, residual_out=None):
    """``rmsnorm`` with each row in 8 bits: returns (q int8 [rows, d], scale fp32
    [rows], x + residual or None); the row is q * scale."""
    residual_out = _norm_args(x, w, residual, residual_out)
    rows, d = x.shape
    q_out = _out("q_out", q_out, x.shape, torch.int8, x)
    scale_out = _out("scale_out", scale_out, (rows,), torch.float32, x)
    rc = L.lib().bllm_rmsnorm_q8(x.data_ptr(), _ptr(residual), w.data_ptr(), _dt(x), rows, d, eps,
                                 _ptr(residual_out), q_out.data_ptr(), scale_out.data_ptr(), _stream())
    L.check("bllm_rmsnorm_q8", rc)
    return q_out, scale_out, residual_out


def quant_rows_q8(x, *, q_out=None, scale_out=None):
    """Rows of x [rows, d] in 8 bits: returns (q int8, scale fp32 [rows])."""
    _dev(x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    rows, d = x.shape
    q_out = _out("q_out", q_out, x.shape, torch.int8, x)
    scale_out = _out("scale_out", scale_out, (rows,), torch.float32, x)
    rc = L.lib().bllm_quant_rows_q8(x.data_ptr(), _dt(x), rows, d, q_out.data_ptr(), scale_out.data_ptr(), _stream())
    L.check("bllm_quant_rows_q8", rc)
    return q_out, scale_out


def linear_i8(xq, x_scale, wq, w_scale, *, bias=None, out_dtype=torch.bfloat16, y_out=None):
    """y [m, n] = (xq @ wq.T) * x_scale[:, None] * w_scale + bias for int8 xq [m, k]
    and wq [n, k], exact integer sums, rounded once to out_dtype (y_out's dtype if given)."""
    if xq.dtype != torch.int8 or wq.dtype != torch.int8:
        raise TypeError("xq and wq must be int8")
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError("xq must be [m, k] and wq [n, k]")
    _dev(xq, wq)
    m, k = xq.shape
    n = wq.shape[0]
    _is("x_scale", x_scale, (m,), torch.float32)
    _is("w_scale", w_scale, (n,), torch.float32)
    if bias is not None:
        _is("bias", bias, (n,), torch.float32)
    y_out = _out("y_out", y_out, (m, n), out_dtype if y_out is None else y_out.dtype, xq)
    rc = L.lib().bllm_linear_i8(xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                                _dt(y_out), m, n, k, y_out.data_ptr(), _stream())
    L.check("bllm_linear_i8", rc)
    return y_out


def _token_stride(name, t, total, heads, width):
    """Distance between tokens of t [total, heads, width], whose heads are dense."""
    if t.shape != (total, heads, width):
        raise ValueError(f"{name} must be [{total}, {heads}, {width}], got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    s0, s1, s2 = t.stride()
    if (width > 1 and s2 != 1) or (heads > 1 and s1 != width):
        raise ValueError(f"the heads of a token of {name} must be dense")
    return s0 if total > 1 else heads * width


def _delta_args(q, k, v, g, beta, o_out):
    if q.dim() != 3 or v.dim() != 3 or q.shape[0] != v.shape[0]:
        raise ValueError("q, k and v must be [tokens, heads, width] with the same tokens")
    total, hk, dk = q.shape
    _, hv, dv = v.shape
    strides = (_token_stride("q", q, total, hk, dk), _token_stride("k", k, total, hk, dk),
               _token_stride("v", v, total, hv, dv))
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k and v must have one dtype")
    _is("g", g, (total, hv), torch.float32)
    _is("beta", beta, (total, hv), torch.float32)
    o_out = _out("o_out", o_out, v.shape, dt, v)
    return ((q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _dt(q)),
            (hk, hv, dk, dv, *strides), o_out)


def gated_delta(q, k, v, g, beta, offsets, *, scale=None, unit_qk: bool = True, state_in=None, state_out=None,
                want_state=True, o_out=None, ws=None):
    """The gated delta rule over a ragged batch: q, k [total, hk, dk], v [total, hv, dv] (bf16, tokens may
    be strided), g and beta fp32 [total, hv], offsets int64 [nseq + 1].  Returns (o [total, hv, dv],
    state fp32 [nseq, hv, dk, dv] or None); state_out may be state_in (updated in place).  scale
    defaults to dk ** -0.5; unit_qk scales every q and k row to unit length first."""
    if state_out is not None and not want_state:
        raise ValueError("state_out needs want_state")
    ptrs, dims, o_out = _delta_args(q, k, v, g, beta, o_out)
    hk, hv, dk, dv = dims[:4]
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be int64 [nseq + 1]")
    _dev(offsets)
    total, nseq = q.shape[0], offsets.shape[0] - 1
    shape = (nseq, hv, dk, dv)
    if state_in is not None:
        _is("state_in", state_in, shape, torch.float32)
    if not want_state:
        state_out = None
    else:
        state_out = _out("state_out", state_out, shape, torch.float32, q)
    w = _ws(gated_delta_workspace(nseq, total, hv, dk, dv), ws, q.device)
    rc = L.lib().bllm_gated_delta(*ptrs, offsets.data_ptr(), nseq, total, *dims,
                                  dk ** -0.5 if scale is None else scale, 1 if unit_qk else 0, _ptr(state_in),
                                  _ptr(state_out), o_out.data_ptr(), w.data_ptr(), _nbytes(w), _stream())
    L.check("bllm_gated_delta", rc)
    return o_out, state_out


def gated_delta_step(q, k, v, g, beta, state, *, state_out=None, slots=None, scale=None, unit_qk: bool = True,
                     o_out=None):
    """One token of each stream: q, k [nseq, hk, dk], v [nseq, hv, dv], g and beta [nseq, hv].  state
    fp32 [nslots, hv, dk, dv] is updated in place unless state_out is given; stream s has row
    slots[s] (int32, row s without slots).  Returns (o [nseq, hv, dv], the state written)."""
    ptrs, dims, o_out = _delta_args(q, k, v, g, beta, o_out)
    hk, hv, dk, dv = dims[:4]
    nseq, nslots = q.shape[0], state.shape[0]
    _is("state", state, (nslots, hv, dk, dv), torch.float32)
    if state_out is None:
        state_out = state
    else:
        _is("state_out", state_out, state.shape, torch.float32)
    if slots is not None:
        _is("slots", slots, (nseq,), torch.int32)
    rc = L.lib().bllm_gated_delta_step(*ptrs, nseq, *dims, dk ** -0.5 if scale is None else scale,
                                       1 if unit_qk else 0, state.data_ptr(), state_out.data_ptr(), _ptr(slots),
                                       nslots, o_out.data_ptr(), _stream())
    L.check("bllm_gated_delta_step", rc)
    return o_out, state_out
