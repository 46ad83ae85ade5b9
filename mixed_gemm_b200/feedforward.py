"""User-facing helpers of the feed-forward operators over the C ABI.

The half of a transformer block around the packed linear: the INT8 product with
a scale per token and per output channel (``quantize_rows_int8``, ``matmul_i8``),
the gated projections (``gated_ff`` and ``gated_ff_backward``) and the norms
around the block (``residual_norm`` and ``residual_norm_backward``).

torch provides device memory and streams; the work runs in ``libwq.so``.  Every
tensor of a call lies on one CUDA device, which need not be the current one.
The call is enqueued on ``stream`` (a ``torch.cuda.Stream`` or a raw
``cudaStream_t``; default: the device's current stream), and what it allocates
(outputs, workspaces) belongs to that stream.  A tensor whose rows are not
contiguous is copied first; outputs are new tensors unless given.  Wrong types,
shapes or devices raise ``ValueError`` before anything is launched, what the
library refuses raises ``WQError``.

``gated_ff`` and ``residual_norm`` are differentiable where an input requires a gradient
(once, not inside CUDA graph capture, and in reverse mode only: a tensor that carries a
forward-mode tangent is refused).  With ``save=True`` they return what the explicit
``..._backward`` calls take and are not recorded by autograd; these forward and backward
calls may be captured into CUDA graphs.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad

from . import ACTIVATIONS, WQ_OK, _lib, _check

_BF16, _F32, _I8 = torch.bfloat16, torch.float32, torch.int8

# The current device and a device's current raw stream, without the wrapper objects (a
# decoded token's calls are bound by the host: the objects cost 3 us a call).
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dual_level():
    # the level of torch.autograd.forward_ad that is entered (-1: none)
    return getattr(forward_ad, "_current_level", 0)


def _no_tangents(where, ts):
    # the kernels see the primal alone: its derivative would read as zero
    for t in ts:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{where} has no forward-mode derivative: a tensor carries a tangent")


def _placed(fn):
    """Runs ``fn(first tensor, ...)`` with the tensor's device and the wanted stream current."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        t = args[0] if args and args[0] is not None else next(
            (a for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{fn.__name__}: CUDA tensors are needed (there is no CPU form)")
        if _dual_level() >= 0:
            _no_tangents(fn.__name__, (*args, *kw.values()))
        if stream is None and t.get_device() == _device():
            return fn(*args, **kw)
        if stream is None:
            stream = torch.cuda.current_stream(t.device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=t.device)
        if stream.device != t.device:
            raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on "
                             f"{t.device}")
        for a in (*args, *kw.values()):  # not to be reused before that stream is done with them
            if isinstance(a, torch.Tensor) and a.is_cuda:
                a.record_stream(stream)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _needs_grad(*ts):
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    return False


def _eager_only(where):
    # A captured backward pass accumulates into leaves whose accumulators an earlier eager
    # graph may have bound to another stream; that ends the process inside the engine.
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{where}: autograd through this call is not captured into CUDA "
                           f"graphs; capture {where}(save=True) and {where}_backward")


_calls = {name: getattr(_lib, name) for name in (
    "wq_quantize_act_int8", "wq_matmul_i8", "wq_gated_ff", "wq_gated_ff_backward",
    "wq_residual_norm", "wq_residual_norm_backward")}


def _run(where, device, *args):
    st = _calls[where](*args, _raw_stream(device))
    if st != WQ_OK:
        _check(st, where)


def _p(t):
    return None if t is None else t.data_ptr()


def _take(where, name, t, dtype, shape, device):
    """``t`` with contiguous rows, checked; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{where}: {name} is {dtype} {list(shape)} on cuda:{device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    return t if t.is_contiguous() else t.contiguous()


def _rows(where, name, t, dtype):
    """[..., n] as [rows, n] with contiguous rows."""
    if t.dtype is not dtype or t.dim() < 1:
        raise ValueError(f"{where}: {name} is {dtype} [..., n], got {t.dtype} {list(t.shape)}")
    if t.dim() != 2:
        n = t.shape[-1]
        t = t.reshape(t.numel() // n if n else 0, n)
    return t if t.is_contiguous() else t.contiguous()


def _output(where, name, out, like, dtype, shape):
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if (out.dtype is not dtype or out.numel() != shape[0] * shape[1] or
            out.shape[-1] != shape[1] or out.device != like.device or not out.is_contiguous()):
        raise ValueError(f"{where}: {name} is a contiguous {dtype} {list(shape)} on {like.device}")
    if _needs_grad(out):
        raise ValueError(f"{where}: {name} is written outside autograd: it must not require a gradient")
    torch.autograd.graph.increment_version(out)  # where a graph has kept it, its use is an error
    return out


def _size(where, *args):
    n = ctypes.c_size_t()
    _check(getattr(_lib, where)(*args, ctypes.byref(n)), where)
    return n.value


@_placed
def quantize_rows_int8(x: torch.Tensor):
    """bf16 [..., K] -> (int8 codes [..., K], fp32 scales [...]): scale = max |x| / 127 of each
    row, codes round half to even (K % 8 == 0).  For activations (a scale per token) and for
    the weight of ``matmul_i8`` (a scale per output channel).  A row with a NaN or an infinity
    gets scale NaN and codes 0.  Neither output has a gradient."""
    if _needs_grad(x):
        raise ValueError("quantize_rows_int8 has no backward pass: detach x")
    rows = _rows("quantize_rows_int8", "x", x, _BF16)
    M, K = rows.shape
    q = rows.new_empty((M, K), dtype=_I8)
    s = rows.new_empty((M,), dtype=_F32)
    _run("wq_quantize_act_int8", rows.get_device(), _p(rows), M, K, _p(q), _p(s))
    return q.view(x.shape), s.view(x.shape[:-1])


@_placed
def matmul_i8(xq: torch.Tensor, sx: torch.Tensor, w: torch.Tensor, sw: torch.Tensor,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              out_dtype: torch.dtype = _BF16) -> torch.Tensor:
    """y = (xq @ w.T) * sx[..., None] * sw + bias with exact integer sums.

    ``xq`` int8 [..., K] and ``sx`` fp32 [...] (a scale per token), ``w`` int8 [N, K] and ``sw``
    fp32 [N] (a scale per output channel), ``bias`` bf16 [N]; K % 16 == 0.  ``out_dtype``:
    bf16 or fp32."""
    f = "matmul_i8"
    x = _rows(f, "xq", xq, _I8)
    M, K = x.shape
    dev = x.get_device()
    if w.dim() != 2:
        raise ValueError(f"{f}: w is int8 [N, K]")
    N = w.shape[0]
    w = _take(f, "w", w, _I8, (N, K), dev)
    sx = _take(f, "sx", sx, _F32, xq.shape[:-1], dev)
    sw = _take(f, "sw", sw, _F32, (N,), dev)
    bias = _take(f, "bias", bias, _BF16, (N,), dev)
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError(f"{f}: out_dtype is bf16 or fp32")
    if _needs_grad(sx, sw, bias):
        raise ValueError(f"{f} has no backward pass: detach sx, sw and bias")
    y = _output(f, "out", out, x, out_dtype, (M, N))
    _run("wq_matmul_i8", dev, x.data_ptr(), sx.data_ptr(), w.data_ptr(), sw.data_ptr(), _p(bias), M,
         N, K, out_dtype is _F32, y.data_ptr())
    return y if xq.dim() == 2 else y.view(*xq.shape[:-1], N)


@_placed
def gated_ff(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
             b_gate: torch.Tensor | None = None, b_up: torch.Tensor | None = None,
             act: str = "silu", save: bool = False, out: torch.Tensor | None = None):
    """h = act(x @ w_gate.T + b_gate) * (x @ w_up.T + b_up) in one kernel, bf16.

    ``x`` [..., K], weights [F, K], biases [F]; ``act``: silu, gelu (exact) or relu; K and F
    multiples of 8.  With ``save`` returns (h, g, u), g and u being the pre-activations
    that ``gated_ff_backward`` takes (and autograd records nothing)."""
    f = "gated_ff"
    if not save and _needs_grad(x, w_gate, w_up, b_gate, b_up):
        if out is not None:
            raise ValueError(f"{f}: out is not for calls that autograd records")
        return _GatedFF.apply(x, w_gate, w_up, b_gate, b_up, act)
    xr = _rows(f, "x", x, _BF16)
    M, K = xr.shape
    dev = xr.get_device()
    if act not in ACTIVATIONS or w_gate.dim() != 2:
        raise ValueError(f"{f}: act is one of {sorted(ACTIVATIONS)}, weights are [F, K]")
    F = w_gate.shape[0]
    w_gate = _take(f, "w_gate", w_gate, _BF16, (F, K), dev)
    w_up = _take(f, "w_up", w_up, _BF16, (F, K), dev)
    b_gate = _take(f, "b_gate", b_gate, _BF16, (F,), dev)
    b_up = _take(f, "b_up", b_up, _BF16, (F,), dev)
    h = _output(f, "out", out, xr, _BF16, (M, F))
    g = u = None
    if save:
        g, u = torch.empty_like(h), torch.empty_like(h)
    _run("wq_gated_ff", dev, xr.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), _p(b_gate),
         _p(b_up), M, F, K, ACTIVATIONS[act], h.data_ptr(), _p(g), _p(u))
    if x.dim() != 2:
        shape = (*x.shape[:-1], F)
        h = h.view(shape)
        if save:
            g, u = g.view(shape), u.view(shape)
    return (h, g, u) if save else h


@_placed
def gated_ff_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                      w_up: torch.Tensor, g: torch.Tensor, u: torch.Tensor, act: str = "silu",
                      need_dx: bool = True, need_dw: bool = True, need_bias: bool = False):
    """Gradients of ``gated_ff`` from dh = dL/dh [..., F] and the kept g, u: (dx, dw_gate, dw_up,
    db_gate, db_up), None for what is not asked for.

    dg and du are rounded to bf16, the operands of the products that make dx and the weights'
    gradients; the bias gradients are sums of the unrounded ones."""
    f = "gated_ff_backward"
    xr = _rows(f, "x", x, _BF16)
    M, K = xr.shape
    dev = xr.get_device()
    if act not in ACTIVATIONS or w_gate.dim() != 2:
        raise ValueError(f"{f}: act is one of {sorted(ACTIVATIONS)}, weights are [F, K]")
    if not (need_dx or need_dw or need_bias):
        return None, None, None, None, None
    F = w_gate.shape[0]
    shape = (*x.shape[:-1], F)
    w_gate = _take(f, "w_gate", w_gate, _BF16, (F, K), dev)
    w_up = _take(f, "w_up", w_up, _BF16, (F, K), dev)
    dh = _take(f, "dh", dh, _BF16, shape, dev)
    g = _take(f, "g", g, _BF16, shape, dev)
    u = _take(f, "u", u, _BF16, shape, dev)
    n = _size("wq_gated_ff_backward_workspace_size", M, F, K, need_bias)
    ws = xr.new_empty((max(n, 16),), dtype=torch.uint8)
    dx = torch.empty_like(xr) if need_dx else None
    dwg = dwu = dbg = dbu = None
    if need_dw:
        dwg, dwu = torch.empty_like(w_gate), torch.empty_like(w_up)
    if need_bias:
        dbg, dbu = xr.new_empty((F,)), xr.new_empty((F,))
    _run("wq_gated_ff_backward", dev, dh.data_ptr(), xr.data_ptr(), w_gate.data_ptr(),
         w_up.data_ptr(), g.data_ptr(), u.data_ptr(), M, F, K, ACTIVATIONS[act], ws.data_ptr(), n,
         _p(dx), _p(dwg), _p(dwu), _p(dbg), _p(dbu))
    return (dx if dx is None or x.dim() == 2 else dx.view(x.shape)), dwg, dwu, dbg, dbu


class _GatedFF(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, b_gate, b_up, act):
        _eager_only("gated_ff")
        h, g, u = gated_ff(x, w_gate, w_up, b_gate, b_up, act=act, save=True)
        ctx.save_for_backward(x, w_gate, w_up, g, u)
        ctx.act = act
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        _eager_only("gated_ff")
        need = ctx.needs_input_grad
        dx, dwg, dwu, dbg, dbu = gated_ff_backward(
            dh, *ctx.saved_tensors, act=ctx.act, need_dx=need[0], need_dw=need[1] or need[2],
            need_bias=need[3] or need[4])
        return dx, *(d if n else None for d, n in zip((dwg, dwu, dbg, dbu), need[1:5])), None


def _gate(f, gate, rows_per_gate, M, D, dev):
    """The gate as [G, D], and the tokens that share a row of it."""
    if gate is None:
        return None, 1
    if gate.dim() < 1 or gate.shape[-1] != D:
        raise ValueError(f"{f}: gate is {_BF16} [..., {D}], got {list(gate.shape)}")
    if gate.dim() != 2:
        gate = gate.reshape(-1, D)
    if rows_per_gate is None:
        if M and (gate.shape[0] == 0 or M % gate.shape[0]):
            raise ValueError(f"{f}: {M} tokens do not divide over {gate.shape[0]} gate rows: "
                             "give rows_per_gate")
        rows_per_gate = max(1, M // max(1, gate.shape[0]))
    per = int(rows_per_gate)
    if per < 1:
        raise ValueError(f"{f}: rows_per_gate is at least 1")
    if M == 0:
        return gate, per
    return _take(f, "gate", gate, _BF16, (-(-M // per), D), dev), per


@_placed
def residual_norm(x: torch.Tensor, y: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                  w_pre: torch.Tensor | None = None, rows_per_gate: int | None = None,
                  scale: float = 1.0, eps: float = 1e-6, quantize: bool = False,
                  save: bool = False, out: torch.Tensor | None = None):
    """The norms after one block and before the next, with the gate, the residual scale and the
    residual sum between them, in one pass:

        r = x + scale * gate * norm(y; w_post)        h = norm(r; w_pre)

    (norm: root mean square).  ``x`` and ``y`` bf16 [..., D], the residual stream and the block's
    output; without ``y`` r is x.  ``w_post`` None: y is taken as it is; ``w_pre`` None: no h.
    ``gate`` bf16 [G, D]: token m takes row m // rows_per_gate (default: the tokens divided
    evenly over the rows).  D % 8 == 0, at most 16384.

    Returns (r, h), or with ``quantize`` (r, codes, scales): h as int8 codes with a scale per
    token, what ``matmul_i8`` takes.  With ``save`` two more, the kept 1 / rms of y and of r
    (fp32, None without the weight) for ``residual_norm_backward`` (and autograd records
    nothing).  ``out`` receives r and may be x itself."""
    f = "residual_norm"
    if not save and _needs_grad(x, y, gate, w_post, w_pre):
        if out is not None or quantize:
            raise ValueError(f"{f}: out and quantize are not for calls that autograd records")
        r, h = _ResidualNorm.apply(x, y, gate, w_post, w_pre, rows_per_gate, scale, eps)
        return (x if y is None else r), h
    xr = _rows(f, "x", x, _BF16)
    M, D = xr.shape
    dev, shape = xr.get_device(), x.shape
    yr = _take(f, "y", y, _BF16, shape, dev)
    w_post = _take(f, "w_post", w_post, _BF16, (D,), dev)
    w_pre = _take(f, "w_pre", w_pre, _BF16, (D,), dev)
    gate, per = _gate(f, gate, rows_per_gate, M, D, dev)
    if quantize and w_pre is None:
        raise ValueError(f"{f}: quantize needs w_pre")
    if out is not None and y is None:
        raise ValueError(f"{f}: out receives r, which is x itself without y")
    r = h = q = s = rp = rn = None
    if y is not None:
        r = torch.empty_like(xr) if out is None else _output(f, "out", out, xr, _BF16, (M, D))
    if w_pre is not None:
        if quantize:
            q = xr.new_empty((M, D), dtype=_I8)
            s = xr.new_empty((M,), dtype=_F32)
        else:
            h = torch.empty_like(xr)
    if save:
        if w_post is not None:
            rp = xr.new_empty((M,), dtype=_F32)
        if w_pre is not None:
            rn = xr.new_empty((M,), dtype=_F32)
    _run("wq_residual_norm", dev, xr.data_ptr(), _p(yr), _p(gate), _p(w_post), _p(w_pre), M, D, per,
         scale, eps, _p(r), _p(h), _p(q), _p(s), _p(rp), _p(rn))
    if len(shape) != 2:
        r, h, q = (None if t is None else t.view(shape) for t in (r, h, q))
        s = None if s is None else s.view(shape[:-1])
    r = x if r is None else r
    got = (r, q, s) if quantize else (r, h)
    return (*got, rp, rn) if save else got


@_placed
def residual_norm_backward(dr: torch.Tensor | None, dh: torch.Tensor | None, x: torch.Tensor,
                           y: torch.Tensor | None, gate: torch.Tensor | None,
                           w_post: torch.Tensor | None, w_pre: torch.Tensor | None,
                           rstd_post: torch.Tensor | None, rstd_pre: torch.Tensor | None,
                           rows_per_gate: int | None = None, scale: float = 1.0):
    """Gradients of ``residual_norm`` from dr = dL/dr and dh = dL/dh (either may be None, not
    both): (dx, dy, dgate, dw_post, dw_pre), None for an input that was None.  ``x`` is the
    forward pass's input (not r, should r have been written over it)."""
    f = "residual_norm_backward"
    xr = _rows(f, "x", x, _BF16)
    M, D = xr.shape
    dev, shape = xr.get_device(), x.shape
    yr = _take(f, "y", y, _BF16, shape, dev)
    dr = _take(f, "dr", dr, _BF16, shape, dev)
    if dr is None and dh is None:
        raise ValueError(f"{f}: dr or dh is needed")
    w_post = _take(f, "w_post", w_post, _BF16, (D,), dev)
    wn = _take(f, "w_pre", w_pre, _BF16, (D,), dev)
    dw_pre = None
    if dh is None:                       # no gradient through h
        if wn is not None:
            dw_pre = torch.zeros_like(wn)
        wn, rstd_pre = None, None
    dh = _take(f, "dh", dh, _BF16, shape, dev)
    rstd_post = _take(f, "rstd_post", rstd_post, _F32, (M,), dev)
    rstd_pre = _take(f, "rstd_pre", rstd_pre, _F32, (M,), dev)
    gate_shape = None if gate is None else gate.shape
    gate, per = _gate(f, gate, rows_per_gate, M, D, dev)
    if y is None and wn is None:         # r is x, and nothing follows
        return dr.clone().view(shape), None, None, None, dw_pre
    n = _size("wq_residual_norm_backward_workspace_size", M, D)
    ws = xr.new_empty((max(n, 16),), dtype=torch.uint8)
    dx = torch.empty_like(xr)
    dy = None if y is None else torch.empty_like(xr)
    dgate = None if gate is None else torch.empty_like(gate) if M else torch.zeros_like(gate)
    dw_post = None if w_post is None else torch.empty_like(w_post)
    if wn is not None:
        dw_pre = torch.empty_like(wn)
    _run("wq_residual_norm_backward", dev, _p(dr), _p(dh), xr.data_ptr(), _p(yr), _p(gate),
         _p(w_post), _p(wn), _p(rstd_post), _p(rstd_pre), M, D, per, scale, ws.data_ptr(), n,
         dx.data_ptr(), _p(dy), _p(dgate), _p(dw_post), None if wn is None else _p(dw_pre))
    if len(shape) != 2:
        dx = dx.view(shape)
        dy = None if dy is None else dy.view(shape)
    if dgate is not None and dgate.shape != gate_shape:
        dgate = dgate.view(gate_shape)
    return dx, dy, dgate, dw_post, dw_pre


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, gate, w_post, w_pre, rows_per_gate, scale, eps):
        _eager_only("residual_norm")
        r, h, rp, rn = residual_norm(x, y, gate, w_post, w_pre, rows_per_gate=rows_per_gate,
                                     scale=scale, eps=eps, save=True)
        ctx.save_for_backward(x, y, gate, w_post, w_pre, rp, rn)
        ctx.rest = rows_per_gate, scale
        ctx.set_materialize_grads(False)
        return (None if y is None else r), h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dr, dh):
        _eager_only("residual_norm")
        if dr is None and dh is None:
            return (None,) * 8
        per, scale = ctx.rest
        got = residual_norm_backward(dr, dh, *ctx.saved_tensors, rows_per_gate=per, scale=scale)
        return *(d if n else None for d, n in zip(got, ctx.needs_input_grad)), None, None, None
