"""Tensor-level helpers over the C ABI: PyTorch allocates device memory and
supplies the stream; the library's kernels do all the arithmetic.

    y, z = monarch_forward(x, w1, w2)              # x [B, in], w1 [b1, q1o, q1i], w2 [b2, q2o, q2i]
    dx, dw1, dw2 = monarch_backward(dy, x, w1, w2, z)

MonarchLinearFunction wraps the pair as an autograd function, so the operator
can stand in for a dense linear layer. The *_ex helpers and the MonarchLinear
module take the general layer (any in/out, zero-padded to whole blocks, an
explicit intermediate width, optional bias).

Around and after the layers: sandwich_forward / sandwich_backward (SandwichNorm)
for the norms, gate and residual join between two blocks, and distill_forward /
distill_backward / distill_step (DistillLossFunction) for training against a
teacher's top logits; head_loss_forward / head_loss_backward / head_loss_step (HeadLossFunction) for
the same loss, or the cross entropy, from a dense head's input without its logits; dropout_forward /
dropout_backward (Dropout) for dropout at a residual join, without a stored mask.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import binding as B


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return B.F32
    if t.dtype == torch.bfloat16:
        return B.BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _expect(t, shape, name: str):
    """Raise ValueError unless tensor t (if given) has exactly this shape; the
    kernels derive every extent from the sizes passed to the library, so a
    tensor of another shape would be read or written out of its bounds."""
    if t is None:
        return
    if tuple(t.shape) != tuple(int(v) for v in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def problem_of(x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor):
    """(in_features, out_features, nblocks1, nblocks2, batch) from tensor shapes,
    after checking w1 == [b1, out/b1, in/b1] and w2 == [b2, out/b2, out/b2]
    (mid = out)."""
    if x.dim() != 2 or w1.dim() != 3 or w2.dim() != 3:
        raise ValueError("x must be [batch, in], w1 [b1, q1o, q1i], w2 [b2, q2o, q2i]")
    nb1, nb2 = int(w1.shape[0]), int(w2.shape[0])
    fi, fo, b = int(x.shape[1]), nb2 * int(w2.shape[1]), int(x.shape[0])
    if nb1 <= 0 or nb2 <= 0 or fi % nb1 or fo % nb1:
        raise ValueError(f"in={fi} and out={fo} must be divisible by nblocks1={nb1}")
    _expect(w1, (nb1, fo // nb1, fi // nb1), "w1")
    _expect(w2, (nb2, fo // nb2, fo // nb2), "w2")
    return fi, fo, nb1, nb2, b


def _check(*ts):
    dt = ts[0].dtype
    for t in ts:
        if t is None:
            continue
        if t.dtype != dt:
            raise TypeError("all tensors must share one dtype")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if t.device.type != "cuda":
            raise ValueError("tensors must live on the GPU")


def _whole(t):
    """t as the library takes it: contiguous, and at a 16-byte boundary (a slice of odd rows is not)."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class _NoSecondDerivative(torch.autograd.Function):
    """Hands gradients on, and raises where they are differentiated."""

    @staticmethod
    def forward(ctx, *grads):
        return tuple(g.detach() for g in grads)   # no views: optimizers write to gradients in place

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the library's operators have no second derivatives")


def _first_derivative_only(backward):
    """For a Function's backward that calls the library. With create_graph=True its results would be
    constants to autograd, and a second derivative would lose their part without a word: they get a
    graph that refuses it instead. (once_differentiable does that only where an incoming gradient
    requires a gradient itself, which the ones of a plain sum do not.)"""

    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        at = [i for i, g in enumerate(out) if g is not None]
        guarded = _NoSecondDerivative.apply(*[out[i].detach().requires_grad_() for i in at])
        out = list(out)
        for i, g in zip(at, guarded):
            out[i] = g
        return tuple(out)

    return wrapped


def monarch_forward(x, w1, w2, act: int = B.ACT_NONE, stream=None):
    fi, fo, nb1, nb2, b = problem_of(x, w1, w2)
    _check(x, w1, w2)
    y = torch.empty((b, fo), dtype=x.dtype, device=x.device)
    z = torch.empty((b, fo), dtype=x.dtype, device=x.device)
    B.monarch_fwd(x, w1, w2, y, z, fi, fo, nb1, nb2, b, dtype_code(x), act, stream)
    return y, z


def monarch_backward(dy, x, w1, w2, z, y=None, act: int = B.ACT_NONE, stream=None,
                     workspace: torch.Tensor | None = None):
    fi, fo, nb1, nb2, b = problem_of(x, w1, w2)
    for t, name in ((dy, "dy"), (z, "z"), (y, "y")):
        _expect(t, (b, fo), name)
    if act == B.ACT_RELU and y is None:
        raise ValueError("the ReLU backward needs the forward output y")
    _check(dy, x, w1, w2, z, y)
    code = dtype_code(x)
    dx = torch.empty_like(x)
    dw1 = torch.empty_like(w1)
    dw2 = torch.empty_like(w2)
    need = B.monarch_bwd_workspace_bytes(fi, fo, nb1, nb2, b, code)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    B.monarch_bwd(dy, x, w1, w2, z, y, dx, dw1, dw2, workspace, need, fi, fo, nb1, nb2, b, code,
                  act, stream)
    return dx, dw1, dw2


def monarch_project(m, nblocks1: int, nblocks2: int, max_steps: int = 256, stream=None,
                    with_status: bool = False):
    """Nearest Monarch factors (w1 [b1, b2, in/b1], w2 [b2, out/b2, b1]) of a
    dense [out, in] matrix; needs out = nblocks1 * nblocks2. With with_status,
    also returns the int32 [b1 * b2] per-slice status (element r*b2 + g for
    slice (g, r)): the products with AᵀA it used when converged, else 0."""
    _check(m)
    if m.dim() != 2:
        raise ValueError("m must be [out, in]")
    fo, fi = m.shape
    if nblocks1 <= 0 or nblocks2 <= 0 or fi % nblocks1 or fo % nblocks2:
        raise ValueError("block counts must divide the matrix dimensions")
    w1 = torch.empty((nblocks1, nblocks2, fi // nblocks1), dtype=m.dtype, device=m.device)
    w2 = torch.empty((nblocks2, fo // nblocks2, nblocks1), dtype=m.dtype, device=m.device)
    conv = torch.empty((nblocks1 * nblocks2,), dtype=torch.int32, device=m.device)
    B.monarch_project(m, w1, w2, fi, fo, nblocks1, nblocks2, dtype_code(m), max_steps, conv,
                      stream)
    return (w1, w2, conv) if with_status else (w1, w2)


class MonarchLinearFunction(torch.autograd.Function):
    """y = act(x · Mᵀ) with M the Monarch matrix of (w1, w2); no bias."""

    @staticmethod
    def forward(ctx, x, w1, w2, act: int = B.ACT_NONE):
        x, w1, w2 = _whole(x), _whole(w1), _whole(w2)
        y, z = monarch_forward(x, w1, w2, act)
        ctx.act = act
        ctx.save_for_backward(x, w1, w2, z, y if act == B.ACT_RELU else None)
        return y

    @staticmethod
    @_first_derivative_only
    def backward(ctx, dy):
        x, w1, w2, z, y = ctx.saved_tensors
        dx, dw1, dw2 = monarch_backward(_whole(dy), x, w1, w2, z, y, ctx.act)
        return dx, dw1, dw2, None


def ex_problem(x, w1, w2, out_features: int, bias=None):
    """(in, out, mid, nb1, nb2, batch) of the general layer from tensor shapes,
    after checking w1 == [b1, mid/b1, ceil(in/b1)], w2 == [b2, ceil(out/b2),
    mid/b2] and bias == [out]."""
    if x.dim() != 2 or w1.dim() != 3 or w2.dim() != 3:
        raise ValueError("x must be [batch, in], w1 [b1, q1o, q1i], w2 [b2, q2o, q2i]")
    nb1, q1o = int(w1.shape[0]), int(w1.shape[1])
    nb2 = int(w2.shape[0])
    mid = nb1 * q1o
    fi, fo, b = int(x.shape[1]), int(out_features), int(x.shape[0])
    if nb1 <= 0 or nb2 <= 0 or fi <= 0 or fo <= 0 or mid % nb2:
        raise ValueError(f"mid={mid} must be divisible by nblocks2={nb2}; sizes must be positive")
    _expect(w1, (nb1, q1o, _cdiv(fi, nb1)), "w1")
    _expect(w2, (nb2, _cdiv(fo, nb2), mid // nb2), "w2")
    if bias is not None and (bias.dim() != 1 or bias.numel() != fo):
        raise ValueError(f"bias has shape {tuple(bias.shape)}, expected ({fo},)")
    return fi, fo, mid, nb1, nb2, b


def monarch_forward_ex(x, w1, w2, out_features: int, bias=None, act: int = B.ACT_NONE,
                       stream=None):
    """y = act(pad(x) · Mᵀ truncated to out_features + bias); returns (y, z)."""
    fi, fo, mid, nb1, nb2, b = ex_problem(x, w1, w2, out_features, bias)
    _check(x, w1, w2, bias)
    y = torch.empty((b, fo), dtype=x.dtype, device=x.device)
    z = torch.empty((b, mid), dtype=x.dtype, device=x.device)
    B.monarch_fwd_ex(x, w1, w2, bias, y, z, fi, fo, mid, nb1, nb2, b, dtype_code(x), act, stream)
    return y, z


def monarch_backward_ex(dy, x, w1, w2, z, y=None, with_bias: bool = False,
                        act: int = B.ACT_NONE, stream=None):
    """(dx, dw1, dw2, dbias or None) of the general layer."""
    if dy.dim() != 2:
        raise ValueError("dy must be [batch, out]")
    fi, fo, mid, nb1, nb2, b = ex_problem(x, w1, w2, dy.shape[1])
    _expect(dy, (b, fo), "dy")
    _expect(y, (b, fo), "y")
    _expect(z, (b, mid), "z")
    if act == B.ACT_RELU and y is None:
        raise ValueError("the ReLU backward needs the forward output y")
    _check(dy, x, w1, w2, z, y)
    code = dtype_code(x)
    dx = torch.empty_like(x)
    dw1 = torch.empty_like(w1)
    dw2 = torch.empty_like(w2)
    db = torch.empty((fo,), dtype=x.dtype, device=x.device) if with_bias else None
    need = B.monarch_bwd_ex_workspace_bytes(fi, fo, mid, nb1, nb2, b, code, with_bias)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    B.monarch_bwd_ex(dy, x, w1, w2, z, y, dx, dw1, dw2, db, ws, need, fi, fo, mid, nb1, nb2, b,
                     code, act, stream)
    return dx, dw1, dw2, db


class MonarchLinearExFunction(torch.autograd.Function):
    """y = act(pad(x) · Mᵀ truncated to out_features + bias)."""

    @staticmethod
    def forward(ctx, x, w1, w2, bias, out_features: int, act: int = B.ACT_NONE):
        x, w1, w2 = _whole(x), _whole(w1), _whole(w2)
        bias = _whole(bias)
        y, z = monarch_forward_ex(x, w1, w2, out_features, bias, act)
        ctx.act = act
        ctx.with_bias = bias is not None
        ctx.save_for_backward(x, w1, w2, z, y if act == B.ACT_RELU else None)
        return y

    @staticmethod
    @_first_derivative_only
    def backward(ctx, dy):
        x, w1, w2, z, y = ctx.saved_tensors
        dx, dw1, dw2, db = monarch_backward_ex(_whole(dy), x, w1, w2, z, y, ctx.with_bias, ctx.act)
        return dx, dw1, dw2, db, None, None


class MonarchLinear(torch.nn.Module):
    """Drop-in for a dense linear layer with the MonarchLinear sizes of the
    "Definition C.3" thread of the scatterbrain issues page: block sizes
    ceil(in/nblocks) and ceil(out/nblocks), intermediate width in_ext for an
    expanding layer and out_ext otherwise; the input is zero-padded to whole
    blocks and the output keeps the first out_features. Optional bias and
    fused ReLU (act)."""

    def __init__(self, in_features: int, out_features: int, nblocks: int = 4, bias: bool = True,
                 act: int = B.ACT_NONE, device=None, dtype=torch.float32):
        super().__init__()
        self.in_features, self.out_features, self.nblocks, self.act = (
            in_features, out_features, nblocks, act)
        mid = B.monarch_linear_mid(in_features, out_features, nblocks)
        q1i = -(-in_features // nblocks)
        q2o = -(-out_features // nblocks)
        self.mid = mid
        self.w1 = torch.nn.Parameter(torch.empty((nblocks, mid // nblocks, q1i), device=device,
                                                 dtype=dtype))
        self.w2 = torch.nn.Parameter(torch.empty((nblocks, q2o, mid // nblocks), device=device,
                                                 dtype=dtype))
        self.bias = (torch.nn.Parameter(torch.empty(out_features, device=device, dtype=dtype))
                     if bias else None)
        self.reset_parameters()

    @torch.no_grad()
    def reset_parameters(self):
        # each factor block is a small dense layer: uniform(+-1/sqrt(fan_in))
        for w in (self.w1, self.w2):
            bound = w.shape[2] ** -0.5
            w.uniform_(-bound, bound)
        if self.bias is not None:
            self.bias.uniform_(-self.in_features ** -0.5, self.in_features ** -0.5)

    def forward(self, x):
        shape = x.shape
        y = MonarchLinearExFunction.apply(x.reshape(-1, shape[-1]), self.w1, self.w2, self.bias,
                                          self.out_features, self.act)
        return y.reshape(*shape[:-1], self.out_features)


def _hyper_shapes(x, ws, dims):
    """Check x == [batch, N] and ws[j] == [N/n_j, n_j, n_j] (N = prod dims)."""
    dims = [int(d) for d in dims]
    if x.dim() != 2 or len(ws) != len(dims) or not dims or min(dims) <= 0:
        raise ValueError("x must be [batch, N] with one weight tensor per lattice axis")
    n = 1
    for d in dims:
        n *= d
    _expect(x, (x.shape[0], n), "x")
    for j, (w, d) in enumerate(zip(ws, dims)):
        _expect(w, (n // d, d, d), f"ws[{j}]")
    return int(x.shape[0]), n


def hyper_forward(x, ws, dims, stream=None):
    """k-factor (hypercube) layer: x [batch, N], ws[j] [N/n_j, n_j, n_j];
    returns (y, saved)."""
    b, n = _hyper_shapes(x, ws, dims)
    _check(x, *ws)
    saved = torch.empty((max(B.monarch_hyper_saved_elems(dims, b), 1),), dtype=x.dtype,
                        device=x.device)
    y = torch.empty_like(x)
    B.monarch_hyper_fwd(x, ws, y, saved, dims, b, dtype_code(x), stream)
    return y, saved


def hyper_backward(dy, x, ws, saved, dims, stream=None):
    """(dx, [dw_j]) of the hypercube layer."""
    b, n = _hyper_shapes(x, ws, dims)
    _expect(dy, (b, n), "dy")
    if saved.numel() < B.monarch_hyper_saved_elems(dims, b):
        raise ValueError("saved is smaller than the forward pass writes")
    _check(dy, x, *ws)
    code = dtype_code(x)
    dx = torch.empty_like(x)
    dws = [torch.empty_like(w) for w in ws]
    need = B.monarch_hyper_bwd_workspace_bytes(dims, b, code)
    ws_buf = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    B.monarch_hyper_bwd(dy, x, ws, saved, dx, dws, ws_buf, need, dims, b, code, stream)
    return dx, dws


def _dyad_shapes(x, wa, wb):
    """Check wb == wa == [nb, qo, qi] and x == [batch, nb*qi]."""
    if x.dim() != 2 or wa.dim() != 3:
        raise ValueError("x must be [batch, in], wa and wb [nb, out/nb, in/nb]")
    nb, qo, qi = (int(v) for v in wa.shape)
    _expect(wb, (nb, qo, qi), "wb")
    _expect(x, (x.shape[0], nb * qi), "x")
    return nb, qo, qi, int(x.shape[0])


def dyad_forward(x, wa, wb, stream=None):
    """DYAD-style layer: y = x · (BD(A) + Q·BD(B)·P)ᵀ; wa, wb [nb, out/nb, in/nb]."""
    nb, qo, qi, b = _dyad_shapes(x, wa, wb)
    _check(x, wa, wb)
    y = torch.empty((b, nb * qo), dtype=x.dtype, device=x.device)
    need = B.monarch_dyad_fwd_workspace_bytes(x.shape[1], nb * qo, nb, b, dtype_code(x))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    B.monarch_dyad_fwd(x, wa, wb, y, ws, need, x.shape[1], nb * qo, nb, b, dtype_code(x), stream)
    return y


def dyad_backward(dy, x, wa, wb, stream=None):
    """(dx, dwa, dwb) of the DYAD-style layer."""
    nb, qo, qi, b = _dyad_shapes(x, wa, wb)
    _expect(dy, (b, nb * qo), "dy")
    _check(dy, x, wa, wb)
    code = dtype_code(x)
    dx, dwa, dwb = torch.empty_like(x), torch.empty_like(wa), torch.empty_like(wb)
    need = B.monarch_dyad_bwd_workspace_bytes(x.shape[1], nb * qo, nb, b, code)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    B.monarch_dyad_bwd(dy, x, wa, wb, dx, dwa, dwb, ws, need, x.shape[1], nb * qo, nb, b, code,
                       stream)
    return dx, dwa, dwb


class SandwichGrads(NamedTuple):
    """Gradients of sandwich_forward's inputs; None where there is no such input."""
    dh: torch.Tensor
    dy: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dpost_bias: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dpre_bias: Optional[torch.Tensor]


def _refuse(t, name, shape, dtype):
    """Raises for the first thing that _beside found wrong with t."""
    _expect(t, shape, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must live on the current GPU, where the call's stream is")


def _saved(stats, shape, dtype, device):
    """Checks what a forward call saved for its backward call."""
    if stats.dtype is not dtype:
        raise ValueError(f"stats must be the {dtype} tensor the forward returned")
    _beside(device, dtype, shape, "stats", stats)


def _beside(device, dtype, shape, names, *tensors):
    """Checks that each given tensor has this dtype and shape, is contiguous and
    lives on GPU `device`; `names` (divided by spaces) are for the refusal."""
    for t in tensors:
        if t is not None and not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and
                                  t.get_device() == device):
            at = next(i for i, x in enumerate(tensors) if x is t)
            _refuse(t, names.split()[at], shape, dtype)


def _sandwich_shapes(h, y, post_weight, post_bias, gate, pre_weight, pre_bias, pre_norm, skip_scale):
    """(rows, features, gates, device) after checking every tensor against h [rows, features]."""
    if h.dim() != 2:
        raise ValueError("h must be [rows, features]")
    rows, d = h.shape
    dtype, device = h.dtype, B.current_device()
    _beside(device, dtype, (rows, d), "h y", h, y)
    _beside(device, dtype, (d,), "post_weight post_bias pre_weight pre_bias", post_weight, post_bias,
            pre_weight, pre_bias)
    gates = 0
    if gate is not None:
        gates = gate.shape[0] if gate.dim() == 2 else -1
        # no rows: any number of gate rows, none too
        if gates < 0 or (rows and (gates == 0 or rows % gates)):
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected (gates, {d}) with gates "
                             f"dividing {rows} rows")
        _beside(device, dtype, (gates, d), "gate", gate)
    if y is None and (post_weight is not None or post_bias is not None or gate is not None or
                      skip_scale != 1.0):
        raise ValueError("without y there is nothing to scale, gate or norm after the block")
    if pre_norm == B.NORM_NONE and (pre_weight is not None or pre_bias is not None):
        raise ValueError("pre_weight and pre_bias need a pre_norm")
    return rows, d, gates, device


def _on_stream(stream, call, *args, **kw):
    """call(*args, **kw) on a stream of the caller's: results and workspaces come
    from that stream's memory, so that none is handed out again before its work is done."""
    if not isinstance(stream, torch.cuda.Stream):
        # 0 is the default stream's handle; ExternalStream(0) would be a stream of torch's own pool
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return call(*args, **kw)


# a function of the sizes alone: asked for once for each of them
_sandwich_workspace = functools.lru_cache(maxsize=256)(B.monarch_sandwich_bwd_workspace_bytes)


def _sandwich_stats(rows, d, y, pre_norm, dtype):
    """(shape, dtype) of stats, monarch_sandwich_stats_bytes long."""
    if y is None or pre_norm == B.NORM_NONE or dtype != torch.bfloat16:
        return (rows, 4), torch.float32
    return (rows, 4 + _cdiv(d, 8)), torch.int32


def sandwich_forward(h, y=None, post_weight=None, post_bias=None, gate=None, pre_weight=None,
                     pre_bias=None, *, post_norm: int = B.NORM_RMS, pre_norm: int = B.NORM_RMS,
                     skip_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-5,
                     stream=None):
    """(h_out, n, stats) of the residual stream h and a block's output y:

        h_out = skip_scale * h + branch_scale * gate * (norm_post(y) * post_weight + post_bias)
        n     = norm_pre(h_out) * pre_weight + pre_bias

    gate [gates, features] holds one row for rows/gates consecutive rows. Without
    y, h_out is h itself (the norm before the first block); with pre_norm
    NORM_NONE, n is None. stats goes to sandwich_backward: fp32 [rows, 4], and in bf16
    with y and a pre_norm int32 [rows, 4 + ceil(features / 8)], which also holds four more
    bits of every value of h_out than its rounding does."""
    if stream is not None:
        return _on_stream(stream, sandwich_forward, h, y, post_weight, post_bias, gate,
                          pre_weight, pre_bias, post_norm=post_norm, pre_norm=pre_norm,
                          skip_scale=skip_scale, branch_scale=branch_scale, eps=eps)
    rows, d, gates, _ = _sandwich_shapes(h, y, post_weight, post_bias, gate, pre_weight, pre_bias,
                                         pre_norm, skip_scale)
    h_out = torch.empty_like(h) if y is not None else h
    n = torch.empty_like(h) if pre_norm != B.NORM_NONE else None
    shape, kind = _sandwich_stats(rows, d, y, pre_norm, h.dtype)
    stats = torch.empty(shape, dtype=kind, device=h.device)
    B.monarch_sandwich_fwd(h, y, post_weight, post_bias, gate, pre_weight, pre_bias,
                           h_out if y is not None else None, n, stats, rows, d, gates, post_norm,
                           pre_norm, skip_scale, branch_scale, eps, dtype_code(h))
    return h_out, n, stats


def sandwich_backward(dh_out, dn, h_out, y, stats, post_weight=None, post_bias=None, gate=None,
                      pre_weight=None, pre_bias=None, *, post_norm: int = B.NORM_RMS,
                      pre_norm: int = B.NORM_RMS, skip_scale: float = 1.0,
                      branch_scale: float = 1.0, stream=None, eps: float | None = None):
    """SandwichGrads from the gradients dh_out (None: zero) and dn of the
    forward's results. h_out and stats are the forward's (eps is in stats; it is
    accepted so that both calls take the same keywords)."""
    if stream is not None:
        return _on_stream(stream, sandwich_backward, dh_out, dn, h_out, y, stats, post_weight,
                          post_bias, gate, pre_weight, pre_bias, post_norm=post_norm,
                          pre_norm=pre_norm, skip_scale=skip_scale, branch_scale=branch_scale)
    if pre_norm != B.NORM_NONE and (dn is None or h_out is None):
        raise ValueError("the backward of a pre_norm needs dn and h_out")
    if pre_norm == B.NORM_NONE and dh_out is None:
        raise ValueError("without a pre_norm the backward needs dh_out")
    ref = h_out if h_out is not None else dh_out
    rows, d, gates, device = _sandwich_shapes(ref, y, post_weight, post_bias, gate, pre_weight,
                                              pre_bias, pre_norm, skip_scale)
    _beside(device, ref.dtype, (rows, d), "dh_out dn", dh_out, dn)
    _saved(stats, *_sandwich_stats(rows, d, y, pre_norm, ref.dtype), device)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    g = SandwichGrads(like(ref), like(y), like(post_weight), like(post_bias), like(gate),
                      like(pre_weight), like(pre_bias))
    code = dtype_code(ref)
    need = _sandwich_workspace(rows, d, gates, post_bias is not None or pre_bias is not None, code)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=ref.device)
    B.monarch_sandwich_bwd(dh_out, dn, h_out, y, stats, post_weight, post_bias, gate, pre_weight,
                           pre_bias, g.dh, g.dy, g.dpost_weight, g.dpost_bias, g.dgate,
                           g.dpre_weight, g.dpre_bias, ws, need, rows, d, gates, post_norm,
                           pre_norm, skip_scale, branch_scale, code)
    return g


class SandwichFunction(torch.autograd.Function):
    """sandwich_forward's (h_out, n) with gradients; n alone without y, None for
    the n of NORM_NONE."""

    @staticmethod
    def forward(ctx, h, y, post_weight, post_bias, gate, pre_weight, pre_bias, how):
        affine = [_whole(t) for t in (post_weight, post_bias, gate, pre_weight, pre_bias)]
        h, y = _whole(h), _whole(y)
        h_out, n, stats = sandwich_forward(h, y, *affine, **how)
        ctx.how, ctx.alone = how, y is None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h_out, y, stats, *affine)
        return n if ctx.alone else (h_out, n)

    @staticmethod
    @_first_derivative_only
    def backward(ctx, *grads):
        h_out, y, stats, *affine = ctx.saved_tensors
        dh_out, dn = (None, grads[0]) if ctx.alone else grads
        if dn is None and ctx.how["pre_norm"] != B.NORM_NONE:
            dn = torch.zeros_like(h_out)
        if dh_out is None and ctx.how["pre_norm"] == B.NORM_NONE:
            dh_out = torch.zeros_like(h_out)
        return (*sandwich_backward(_whole(dh_out), _whole(dn), h_out, y, stats, *affine, **ctx.how), None)


class SandwichNorm(torch.nn.Module):
    """What stands between two blocks: norm, gate and residual join of the first
    one's output, norm for the second one.

        h, n = SandwichNorm(features)(h, y)      # y: the output of a block that read n

    pre_norm NORM_NONE ends the stream without a norm; `gated` adds a learned gate
    row (a gate of the caller's own, [gates, features], may be passed instead)."""

    def __init__(self, features: int, post_norm: int = B.NORM_RMS, pre_norm: int = B.NORM_RMS,
                 bias: bool = False, gated: bool = False, skip_scale: float = 1.0,
                 branch_scale: float = 1.0, eps: float = 1e-5, device=None, dtype=torch.float32):
        super().__init__()
        make = lambda on, v: (torch.nn.Parameter(torch.full((features,), v, device=device, dtype=dtype))  # noqa: E731
                              if on else None)
        self.how = dict(post_norm=post_norm, pre_norm=pre_norm, skip_scale=skip_scale,
                        branch_scale=branch_scale, eps=eps)
        self.post_weight, self.post_bias = make(True, 1.0), make(bias, 0.0)
        self.pre_weight = make(pre_norm != B.NORM_NONE, 1.0)
        self.pre_bias = make(bias and pre_norm != B.NORM_NONE, 0.0)
        self.gate = (torch.nn.Parameter(torch.ones((1, features), device=device, dtype=dtype))
                     if gated else None)

    def forward(self, h, y, gate=None):
        shape = h.shape
        flat = lambda t: t.reshape(-1, shape[-1])  # noqa: E731
        h_out, n = SandwichFunction.apply(flat(h), flat(y), self.post_weight, self.post_bias,
                                          self.gate if gate is None else gate, self.pre_weight,
                                          self.pre_bias, self.how)
        return h_out.reshape(shape), None if n is None else n.reshape(shape)


def _distill_shapes(logits, teacher, ids, labels, per_row, name):
    """(rows, vocab, top, ld, device) after checking logits [rows, vocab] (rows may lie
    apart, columns may not), teacher and ids [rows, top], labels and per_row [rows]."""
    if logits.dim() != 2 or teacher.dim() != 2:
        raise ValueError("logits must be [rows, vocab], the teacher's logits [rows, top]")
    rows, vocab = logits.shape
    top, device = teacher.shape[1], B.current_device()
    if top > B.DISTILL_MAX_TOP:
        raise ValueError(f"at most {B.DISTILL_MAX_TOP} teacher entries a row, got {top}")
    _beside(device, torch.float32, (rows, top), "teacher", teacher)
    _beside(device, torch.int64, (rows, top), "ids", ids)
    _beside(device, torch.int64, (rows,), "labels", labels)
    _beside(device, torch.float32, (rows,), name, per_row)
    if logits.get_device() != device:
        raise ValueError("logits must live on the current GPU, where the call's stream is")
    return rows, vocab, top, _rows_apart(logits, rows, vocab, "logits"), device


def _rows_apart(t, rows, cols, name):
    """Elements from one row of t [rows, cols] to the next."""
    ld = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name} must have rows of side by side columns that do not overlap")
    return ld


def _distill_out(logits, rows, vocab, ld, device, out):
    """(dlogits, its ld): `out` after checking it, or new memory. That has the logits' own
    layout where their rows have little padding (up to an eighth); rows that lie further
    apart (a position of a sequence, every k-th row) are stored side by side, each at the
    offset from a 16-byte boundary that it has in the logits."""
    if out is None:
        if ld - vocab > vocab // 8:
            ld = vocab + (ld - vocab) % (16 // logits.element_size())
        out = torch.empty((rows, ld), dtype=logits.dtype, device=logits.device)
        return (out if ld == vocab else out[:, :vocab]), ld
    _expect(out, (rows, vocab), "out")
    if out.dtype != logits.dtype or out.get_device() != device:
        raise ValueError("out must have the logits' dtype and device")
    dld = _rows_apart(out, rows, vocab, "out")
    # the library writes behind autograd's back: a backward pass that saved out's present values has to raise
    torch.autograd.graph.increment_version(out)
    return out, dld


def distill_forward(logits, teacher, ids, labels=None, *, temperature: float = 1.0,
                    mix: float = 1.0, stream=None):
    """(loss [rows], stats) of distillation from a teacher's top logits:

        loss = mix * temperature^2 * KL(p || softmax(logits / temperature)) + (1 - mix) * CE(labels)

    p = softmax(teacher / temperature) over the row's entries, which sit at the
    columns `ids` (int64; -1 pads, and so do teacher logits that are -inf or NaN). labels (int64) outside the vocabulary are ignored.
    stats goes to distill_backward."""
    if stream is not None:
        return _on_stream(stream, distill_forward, logits, teacher, ids, labels,
                          temperature=temperature, mix=mix)
    rows, vocab, top, ld, _ = _distill_shapes(logits, teacher, ids, labels, None, "")
    loss = torch.empty((rows,), dtype=torch.float32, device=logits.device)
    stats = torch.empty((rows, 4), dtype=torch.float32, device=logits.device)
    B.monarch_distill_fwd(logits, ld, teacher, ids, labels, loss, stats, rows, vocab, top,
                          temperature, mix, dtype_code(logits))
    return loss, stats


def distill_backward(dloss, logits, teacher, ids, labels, stats, *, temperature: float = 1.0,
                     mix: float = 1.0, out=None, stream=None):
    """dlogits for dloss [rows]; out may be logits itself."""
    if stream is not None:
        return _on_stream(stream, distill_backward, dloss, logits, teacher, ids, labels, stats,
                          temperature=temperature, mix=mix, out=out)
    rows, vocab, top, ld, device = _distill_shapes(logits, teacher, ids, labels, dloss, "dloss")
    _saved(stats, (rows, 4), torch.float32, device)
    dz, dld = _distill_out(logits, rows, vocab, ld, device, out)
    B.monarch_distill_bwd(dloss, logits, ld, teacher, ids, labels, stats, dz, dld, rows, vocab, top,
                          temperature, mix, dtype_code(logits))
    return dz


def distill_step(logits, teacher, ids, labels=None, row_weight=None, *, temperature: float = 1.0,
                 mix: float = 1.0, out=None, stream=None):
    """(loss [rows], dlogits) in one pass: dlogits is the gradient of
    sum(row_weight * loss) (row_weight None: 1 for every row). out may be
    logits itself, which saves a tensor of their size (autograd sees that they
    changed: what saved their values for its backward pass raises there)."""
    if stream is not None:
        return _on_stream(stream, distill_step, logits, teacher, ids, labels, row_weight,
                          temperature=temperature, mix=mix, out=out)
    rows, vocab, top, ld, device = _distill_shapes(logits, teacher, ids, labels, row_weight,
                                                   "row_weight")
    loss = torch.empty((rows,), dtype=torch.float32, device=logits.device)
    dz, dld = _distill_out(logits, rows, vocab, ld, device, out)
    B.monarch_distill_step(logits, ld, teacher, ids, labels, row_weight, loss, dz, dld, rows, vocab,
                           top, temperature, mix, dtype_code(logits))
    return loss, dz


class DistillLossFunction(torch.autograd.Function):
    """distill_forward's loss with its gradient by the logits, for logits [..., vocab], teacher
    and ids [..., top] and labels [...]: one loss a row, [...]. What does not lie as the
    library takes it is copied. Where the rows' weights are known before the loss,
    distill_step is one pass instead of two."""

    @staticmethod
    def forward(ctx, logits, teacher, ids, labels, temperature: float = 1.0, mix: float = 1.0):
        lead = logits.shape[:-1]
        for t, shape, name in ((teacher, (*lead, teacher.shape[-1]), "teacher"), (ids, teacher.shape, "ids"),
                               (labels, lead, "labels")):
            _expect(t, shape, name)
        flat = lambda t: t.reshape(lead.numel(), t.shape[-1])  # noqa: E731
        z = flat(logits)
        if z.numel() and (z.stride(1) != 1 or z.stride(0) < z.shape[1]):
            z = z.contiguous()
        saved = (z, flat(teacher).contiguous(), flat(ids).contiguous(),
                 None if labels is None else labels.reshape(lead.numel()).contiguous())
        ctx.how = dict(temperature=temperature, mix=mix)
        loss, stats = distill_forward(*saved, **ctx.how)
        ctx.save_for_backward(*saved, stats)
        return loss.view(lead)

    @staticmethod
    @_first_derivative_only
    def backward(ctx, dloss):
        dz = distill_backward(dloss.reshape(-1).contiguous(), *ctx.saved_tensors, **ctx.how)
        return dz.view(*dloss.shape, dz.shape[1]), None, None, None, None, None


def _head_shapes(x, w, labels, teacher, ids, per_row, name):
    """(rows, features, vocab, top, ldx, device) after checking x [rows, features] (rows may lie
    apart), w [vocab, features], labels and per_row [rows], teacher and ids [rows, top]."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [rows, features], w [vocab, features]")
    rows, d = x.shape
    vocab, device = w.shape[0], B.current_device()
    _beside(device, x.dtype, (vocab, d), "w", w)
    if (teacher is None) != (ids is None):
        raise ValueError("teacher and ids come together")
    top = 0
    if teacher is not None:
        top = teacher.shape[1] if teacher.dim() == 2 else -1
        if top < 0 or top > B.DISTILL_MAX_TOP:
            raise ValueError(f"the teacher's logits must be [rows, top], top at most {B.DISTILL_MAX_TOP}")
        _beside(device, torch.float32, (rows, top), "teacher", teacher)
        _beside(device, torch.int64, (rows, top), "ids", ids)
    _beside(device, torch.int64, (rows,), "labels", labels)
    _beside(device, torch.float32, (rows,), name, per_row)
    if x.get_device() != device:
        raise ValueError("x must live on the current GPU, where the call's stream is")
    return rows, d, vocab, top, _rows_apart(x, rows, d, "x"), device


def _teachers_share(mix, teacher):
    """mix, which is 0 without a teacher; with one it has to be given (distill_* take it whole then, a loss of
    labels none of it)."""
    if mix is not None:
        return mix
    if teacher is not None and teacher.numel():
        raise ValueError("a teacher needs mix: its share of the loss, 1 for all of it")
    return 0.0


# a function of the sizes alone: asked for once for each of them
_head_workspace = functools.lru_cache(maxsize=256)(B.monarch_head_workspace_bytes)


def head_loss_forward(x, w, labels=None, teacher=None, ids=None, *, temperature: float = 1.0,
                      mix: Optional[float] = None, stream=None):
    """(loss [rows], stats) of rows x [rows, features] under a dense head w [vocab, features], whose
    logits z = x wᵀ are not kept:

        loss = mix * temperature^2 * KL(p || softmax(z / temperature)) + (1 - mix) * CE(labels)

    with labels, teacher and ids as for distill_forward; without a teacher (or one of no columns), or with
    mix 0, it is the softmax cross entropy. mix has to be given where there is a teacher. Rows without a
    label and a valid entry have loss 0 and cost nothing. stats goes to head_loss_backward."""
    mix = _teachers_share(mix, teacher)
    if stream is not None:
        return _on_stream(stream, head_loss_forward, x, w, labels, teacher, ids,
                          temperature=temperature, mix=mix)
    rows, d, vocab, top, ldx, _ = _head_shapes(x, w, labels, teacher, ids, None, "")
    code = dtype_code(x)
    loss = torch.empty((rows,), dtype=torch.float32, device=x.device)
    stats = torch.empty((rows * (4 + top),), dtype=torch.float32, device=x.device)
    need = _head_workspace(B.HEAD_FWD, rows, d, vocab, top, code)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    B.monarch_head_fwd(x, ldx, w, labels, teacher, ids, loss, stats, ws, need, rows, d, vocab, top,
                       temperature, mix, code)
    return loss, stats


def head_loss_backward(dloss, x, w, labels, teacher, ids, stats, *, temperature: float = 1.0,
                       mix: Optional[float] = None, stream=None):
    """(dx, dw) for dloss [rows]; stats is the forward's. The logits are computed again."""
    mix = _teachers_share(mix, teacher)
    if stream is not None:
        return _on_stream(stream, head_loss_backward, dloss, x, w, labels, teacher, ids, stats,
                          temperature=temperature, mix=mix)
    rows, d, vocab, top, ldx, device = _head_shapes(x, w, labels, teacher, ids, dloss, "dloss")
    _saved(stats, (rows * (4 + top),), torch.float32, device)
    code = dtype_code(x)
    dx = torch.empty((rows, d), dtype=x.dtype, device=x.device)
    dw = torch.empty_like(w)
    need = _head_workspace(B.HEAD_BWD, rows, d, vocab, top, code)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    B.monarch_head_bwd(dloss, x, ldx, w, labels, teacher, ids, stats, dx, dw, ws, need, rows, d, vocab,
                       top, temperature, mix, code)
    return dx, dw


def head_loss_step(x, w, labels=None, teacher=None, ids=None, row_weight=None, *,
                   temperature: float = 1.0, mix: Optional[float] = None, stream=None):
    """(loss [rows], dx, dw) in one call: the gradients of sum(row_weight * loss) (row_weight
    None: 1 for every row). The logits' gradient is held a piece of at most 1 GiB at a time and the logits are
    computed twice: bf16 steps of thousands of rows whose logits fit in memory are a fifth to two fifths slower than
    with the logits kept (a product, distill_step in their place, two products)."""
    mix = _teachers_share(mix, teacher)
    if stream is not None:
        return _on_stream(stream, head_loss_step, x, w, labels, teacher, ids, row_weight,
                          temperature=temperature, mix=mix)
    rows, d, vocab, top, ldx, _ = _head_shapes(x, w, labels, teacher, ids, row_weight, "row_weight")
    code = dtype_code(x)
    loss = torch.empty((rows,), dtype=torch.float32, device=x.device)
    dx = torch.empty((rows, d), dtype=x.dtype, device=x.device)
    dw = torch.empty_like(w)
    need = _head_workspace(B.HEAD_STEP, rows, d, vocab, top, code)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    B.monarch_head_step(x, ldx, w, labels, teacher, ids, row_weight, loss, dx, dw, ws, need, rows, d,
                        vocab, top, temperature, mix, code)
    return loss, dx, dw


class HeadLossFunction(torch.autograd.Function):
    """head_loss_forward's loss with its gradients by x and w, for x [..., features], labels [...],
    teacher and ids [..., top]: one loss a row, [...]. What does not lie as the library takes it is
    copied. Where the rows' weights are known before the loss, head_loss_step computes the logits of
    the backward pass behind those of the forward pass in one call. Both gradients are computed, also
    where only one of x and w needs its own."""

    @staticmethod
    def forward(ctx, x, w, labels, teacher, ids, temperature: float = 1.0, mix: Optional[float] = None):
        lead = x.shape[:-1]
        _expect(labels, lead, "labels")
        if teacher is not None and ids is not None:
            _expect(teacher, (*lead, teacher.shape[-1]), "teacher")
            _expect(ids, teacher.shape, "ids")
        flat = lambda t: None if t is None else t.reshape(lead.numel(), t.shape[-1])  # noqa: E731
        rows = flat(x)
        if rows.numel() and (rows.stride(1) != 1 or rows.stride(0) < rows.shape[1]):
            rows = rows.contiguous()
        whole = lambda t: None if t is None else t.contiguous()  # noqa: E731
        saved = (rows, _whole(w), whole(None if labels is None else labels.reshape(lead.numel())),
                 whole(flat(teacher)), whole(flat(ids)))
        ctx.how, ctx.lead = dict(temperature=temperature, mix=_teachers_share(mix, teacher)), lead
        loss, stats = head_loss_forward(*saved, **ctx.how)
        ctx.save_for_backward(*saved, stats)
        return loss.view(lead)

    @staticmethod
    @_first_derivative_only
    def backward(ctx, dloss):
        dx, dw = head_loss_backward(dloss.reshape(-1).contiguous(), *ctx.saved_tensors, **ctx.how)
        return dx.view(*ctx.lead, dx.shape[1]), dw, None, None, None, None, None


def _dropout_args(p, seed, offset, state, device):
    """(seed, offset) after checking them; p is checked by the library."""
    if state is not None:
        _beside(device, torch.int64, (2,), "state", state)
        return 0, 0
    if seed is None:
        raise ValueError("dropout needs a seed or a state")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be in [0, 2^64)")
    return seed, offset


def dropout_forward(x, p: float, seed: Optional[int] = None, offset: int = 0, residual=None, *,
                    state=None, stream=None):
    """residual + dropout(x) (residual None: dropout(x)) for x and residual of any one shape:

        y = residual + (r >= t ? x / (1 - t / 65536) : 0),    t = round(65536 p)

    r: 16 bits for each element, drawn from (seed, offset) and its place alone, so no mask is kept and
    the backward pass draws them again; give every call an offset of its own. state (int64 [2] on the
    GPU: seed and offset) takes their place where a captured graph draws anew at each replay: the
    program then changes it between replays, and behind the backward pass that draws from it. Calls
    that share a state's value drop the same elements: every call of a step needs a state of its own, for
    instance a row of one [calls, 2] tensor."""
    if stream is not None:
        return _on_stream(stream, dropout_forward, x, p, seed, offset, residual, state=state)
    device = B.current_device()
    _beside(device, x.dtype, x.shape, "x residual", x, residual)
    seed, offset = _dropout_args(p, seed, offset, state, device)
    y = torch.empty_like(x)
    B.monarch_dropout(x, residual, y, x.numel(), p, seed, offset, state, dtype_code(x))
    return y


def dropout_backward(dy, p: float, seed: Optional[int] = None, offset: int = 0, *, state=None,
                     stream=None):
    """dx of dropout_forward's call with the same p, seed and offset (or state); the residual's
    gradient is dy itself."""
    return dropout_forward(dy, p, seed, offset, state=state, stream=stream)


class DropoutFunction(torch.autograd.Function):
    """dropout_forward with gradients by x and the residual. A state's present value is kept for the
    backward pass."""

    @staticmethod
    def forward(ctx, x, p, seed, offset, residual, state):
        ctx.p, ctx.seed, ctx.offset, ctx.joined = p, seed, offset, residual is not None
        ctx.save_for_backward(None if state is None else state.clone())
        return dropout_forward(_whole(x), p, seed, offset, _whole(residual), state=state)

    @staticmethod
    @_first_derivative_only
    def backward(ctx, dy):
        state, = ctx.saved_tensors
        dx = dropout_backward(_whole(dy), ctx.p, ctx.seed, ctx.offset, state=state) if ctx.needs_input_grad[0] else None
        return dx, None, None, None, dy if ctx.joined else None, None


class Dropout(torch.nn.Module):
    """residual + dropout(x) in training, residual + x otherwise. Every call draws anew: under a seed
    that it takes from torch's generator on the CPU, as torch's own dropout takes its numbers. So a copy of the
    module drops elements of its own, a run goes on where the generator's state is restored, and a
    forward pass that is computed again under activation checkpointing, which restores that
    state, drops what the first one dropped.

    With a `seed` of the module's own, call k has offset k (in every module of that seed: a copy drops the
    same elements); the number of calls is kept in the state_dict. A forward pass that is computed
    again would be another call, so one inside a backward pass raises.

    A captured graph would replay one draw: pass a `state` then (dropout_forward), one for every call of a
    step. It takes the place of seed and count, and is not moved on here."""

    def __init__(self, p: float = 0.1, seed: Optional[int] = None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be in [0, 1], got {p}")
        self.p = p
        self.seed = seed
        self.calls = 0

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        if self.seed is not None:
            destination[prefix + "calls"] = torch.tensor(self.calls, device="cpu")

    def _load_from_state_dict(self, state_dict, prefix, *rest):
        # weights saved without a count leave it as it is
        calls = state_dict.pop(prefix + "calls", None)
        if calls is not None and self.seed is not None:
            self.calls = int(calls)
        super()._load_from_state_dict(state_dict, prefix, *rest)

    def forward(self, x, residual=None, state=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else residual + x
        seed, offset = self.seed, self.calls
        if state is None and seed is None:
            seed, offset = int(torch.randint(0, (1 << 63) - 1, (), device="cpu")), 0
        elif state is None and torch._C._current_graph_task_id() != -1:
            raise RuntimeError("Dropout with a seed counts its calls, so a forward pass that is computed again in the backward "
                               "pass (activation checkpointing) would drop other elements: leave the seed out, or pass a state")
        self.calls += 1
        return DropoutFunction.apply(x, self.p, seed, offset, residual, state)
