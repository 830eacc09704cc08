"""Python binding of the source's side of a round: the norm with the residual's
addition, the router's choice, the balance loss, and their gradients.

Argument checks and marshalling only: the arithmetic runs in the HIP library.
rms_norm, route_tokens and balance_loss are differentiable where an input asks
for a gradient; their gradients are also calls of their own (rms_norm_grad,
route_tokens_grad, balance_loss_grad), which is how a captured graph has them.
An output that is given counts as changed in place: a graph that saved it refuses
its backward pass.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _native as nat
from .experts import SCALE_BLOCK, on_device, raw_stream, wrote

_CODES = {torch.bfloat16: nat.AFD_BF16, torch.float32: nat.AFD_FP32}


class Normed(NamedTuple):
    rows: torch.Tensor                # [T, H] bfloat16 or float8_e4m3fn
    scales: Optional[torch.Tensor]    # [T, H/128] float32 (float8 only)
    residual: Optional[torch.Tensor]  # [T, H] the stream, x + residual (None without a residual)
    rstd: Optional[torch.Tensor]      # [T] float32 (with keep_rstd)


class Routes(NamedTuple):
    ids: torch.Tensor      # [T, topk] int32, -1: no expert
    weights: torch.Tensor  # [T, topk] float32


class Balance(NamedTuple):
    loss: torch.Tensor    # [] float32
    counts: torch.Tensor  # [E] int32: choices of every expert
    slope: torch.Tensor   # [E] float32: of the loss by the expert's sum of shares


def _asks(*tensors):
    """Whether a tensor asks for a gradient; what carries a forward one is refused."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("the source's calls have no forward gradients: pass the primal of a dual tensor")
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _plain(call, *tensors):
    if _asks(*tensors):
        raise ValueError(f"{call}: no gradient reaches these arguments: detach them or call under no_grad()")


def _recorded(call, device, *given):
    """A call that autograd records makes its own outputs, and outside of a capture: the backward
    pass of a captured graph meets whatever other graphs hold of the same leaves."""
    if any(given):
        raise ValueError(f"{call}: outputs that are given, and float8 rows, have no gradient: leave them out, or call "
                         f"under no_grad() and {call}_grad for the gradient")
    if device.type == "cuda":
        with on_device(device):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError(f"{call}: autograd does not record a captured call: call it under no_grad(), and "
                                 f"{call}_grad for the gradient")


def _launch(device, call, *args):
    """A call of the library on the device and its current stream."""
    if device.index == torch._C._cuda_getDevice():
        return call(*args, torch._C._cuda_getCurrentRawStream(device.index))
    with on_device(device):
        return call(*args, raw_stream(device))


def _layout(t):
    """What the checks of a tensor look at, but for its address."""
    return t.dtype, t.shape, t.stride(), t.device


_CHECKED = 1024      # layouts of arguments that the calls keep as checked
_norms, _norm_grads, _routes, _balances = {}, {}, {}, {}


def _keep(plans, key, plan):
    if key[1][1] == 1:       # one column: _signed has to look at every call's tensors
        return plan
    if len(plans) >= _CHECKED:
        plans.clear()
    plans[key] = plan
    return plan


def _signed(t, what):
    """The imaginary part of a conjugate is the conjugated memory and a sign beside it.  Its elements
    lie two apart, so that the checks of strides pass those of one element or column alone."""
    if t.is_neg():
        raise ValueError(f"{what}: its sign is not in its memory: call resolve_neg() on it")


def _rows(t, what, device=None):
    """[rows, columns] with its columns next to each other; returns the row stride."""
    if t.dim() != 2 or t.device.type != "cuda" or device is not None and t.device != device or \
            t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must be a [rows, columns] tensor on {device or 'a GPU'} whose columns lie next to each "
                         f"other, got {list(t.shape)} with strides {t.stride()} on {t.device}")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows that share memory (row stride {t.stride(0)} of {t.shape[1]} columns)")
    _signed(t, what)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _wide_rows(t, what, device=None):
    """_rows for a norm: 16-byte pieces."""
    stride = _rows(t, what, device)
    if t.numel() and stride % 8:
        raise ValueError(f"{what} must have a row stride in multiples of 8, got {stride} elements")
    return stride


def _check(status, call, **wide):
    """What the library refused; `wide` tensors lie at multiples of 16 bytes."""
    for what, t in wide.items():
        if t is not None and t.data_ptr() % 16:
            raise ValueError(f"{call}: {what} must be 16-byte aligned")
    nat.check(status, call)


def _like(t, dtype):
    """New contiguous memory of t's shape (from t itself where it is contiguous: half a microsecond less)."""
    if t.is_contiguous():
        return torch.empty_like(t, dtype=dtype)
    return torch.empty(t.shape, dtype=dtype, device=t.device)


def _want(t, what, dtype, shape, device):
    if t is None or t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on {device}, got " + (
            "None" if t is None else f"{t.dtype} {list(t.shape)} on {t.device}, contiguous {t.is_contiguous()}"))
    _signed(t, what)
    return t.data_ptr()


def _code(t, what):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be bfloat16 or float32, got {t.dtype}") from None


@functools.lru_cache(maxsize=256)
def _norm_config(hidden, x, residual, weight, out, eps):
    if not 0 < hidden <= nat.MAX_NORM_HIDDEN or hidden % (SCALE_BLOCK if out == nat.AFD_FP8_E4M3 else 8):
        raise ValueError(f"a norm's columns are a multiple of 8 (of 128 for float8 rows) up to {nat.MAX_NORM_HIDDEN}, got "
                         f"{hidden}")
    if not torch.finfo(torch.float32).tiny <= eps <= torch.finfo(torch.float32).max:
        raise ValueError(f"eps must be a normal positive float32, got {eps}")
    return nat.NormConfig(hidden, x, residual, weight, out, eps)


def _norm_plan(x, weight, residual, eps, dtype, out, out_scales, residual_out):
    """(configuration, strides of x, residual and residual_out) of a norm whose arguments' layouts fit."""
    xs = _wide_rows(x, "x")
    (T, H), dev = x.shape, x.device
    rs, hs, rc = 0, H, nat.NO_RESIDUAL
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError(f"residual must be {list(x.shape)} like x, got {list(residual.shape)}")
        rs, rc = _wide_rows(residual, "residual", dev), _code(residual, "residual")
    if dtype is not torch.bfloat16 and dtype is not torch.float8_e4m3fn:
        raise TypeError(f"dtype must be bfloat16 or float8_e4m3fn, got {dtype}")
    _want(weight, "weight", weight.dtype, (H,), dev)
    cfg = _norm_config(H, _code(x, "x"), rc, _code(weight, "weight"),
                       nat.AFD_BF16 if dtype is torch.bfloat16 else nat.AFD_FP8_E4M3, eps)
    if out is not None:
        _want(out, "out", dtype, (T, H), dev)
    if out_scales is not None:
        if dtype is torch.bfloat16:
            raise ValueError("out_scales belong to float8_e4m3fn rows")
        _want(out_scales, "out_scales", torch.float32, (T, H // SCALE_BLOCK), dev)
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out without a residual")
        if residual_out.dtype is not residual.dtype or residual_out.shape != residual.shape:
            raise ValueError(f"residual_out must be {residual.dtype} {list(residual.shape)} like residual")
        hs = _wide_rows(residual_out, "residual_out", dev)
    return cfg, xs, rs, hs


def _norm(x, weight, residual, eps, dtype, out, out_scales, residual_out, keep_rstd):
    key = (x.dtype, x.shape, x.stride(), x.device, weight.dtype, weight.shape, weight.stride(), weight.device,
           None if residual is None else _layout(residual), eps, dtype, None if out is None else _layout(out),
           None if out_scales is None else _layout(out_scales), None if residual_out is None else _layout(residual_out))
    plan = _norms.get(key) or _keep(_norms, key, _norm_plan(x, weight, residual, eps, dtype, out, out_scales, residual_out))
    cfg, xs, rs, hs = plan
    (T, H), dev = x.shape, x.device
    if out is None:
        out = _like(x, dtype)
    ps = pr = ph = None
    if dtype is torch.float8_e4m3fn:
        if out_scales is None:
            out_scales = torch.empty((T, H // SCALE_BLOCK), dtype=torch.float32, device=dev)
        ps = out_scales.data_ptr()
    if residual is not None:
        if residual_out is None:
            residual_out = _like(residual, residual.dtype)
        pr, ph = residual.data_ptr(), residual_out.data_ptr()
    rstd = torch.empty(T, dtype=torch.float32, device=dev) if keep_rstd else None
    st = _launch(dev, nat.load().afd_norm, cfg, T, x.data_ptr(), xs, pr, rs, weight.data_ptr(), out.data_ptr(), ps, ph, hs,
                 rstd.data_ptr() if keep_rstd else None)
    if st:
        _check(st, "rms_norm", x=x, weight=weight, residual=residual, out=out, residual_out=residual_out)
    return Normed(out, out_scales, residual_out, rstd)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        n = _norm(x, weight, residual, eps, torch.bfloat16, None, None, None, True)
        ctx.set_materialize_grads(False)
        if residual is None or x.requires_grad or residual.requires_grad:
            ctx.mark_non_differentiable(n.rstd)
        else:
            ctx.mark_non_differentiable(n.rstd, n.residual)      # only the weight asks
        ctx.save_for_backward(x if residual is None else n.residual, weight, n.rstd)
        ctx.types = x.dtype, None if residual is None else residual.dtype
        return n.rows, n.residual, n.rstd

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, grad_residual, _):
        if grad is None and grad_residual is None:
            return None, None, None, None
        h, weight, rstd = ctx.saved_tensors
        xt, rt = ctx.types
        dw = None
        if grad is None:
            dh = grad_residual
        else:
            with on_device(h.device):
                if torch.cuda.is_current_stream_capturing():
                    raise ValueError("rms_norm: its backward pass is not captured: call rms_norm_grad")
            dh, dw = rms_norm_grad(_dense(grad), h, weight, rstd,
                                   grad_residual=None if grad_residual is None else _dense(grad_residual),
                                   weight_grad=ctx.needs_input_grad[1])
        return (dh.to(xt) if ctx.needs_input_grad[0] else None, None if dw is None else dw.to(weight.dtype),
                dh if rt is not None and ctx.needs_input_grad[2] else None, None)


def _dense(t):
    """A gradient as autograd hands it on, in memory as the calls take it."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def rms_norm(x, weight, residual=None, *, eps=1e-6, dtype=torch.bfloat16, out=None, out_scales=None, residual_out=None,
             keep_rstd=False) -> Normed:
    """The root-mean-square norm of h = x + residual (or of x), rows y = h / sqrt(mean(h^2) + eps) * weight.

    x [T, H], residual [T, H] and weight [H] are bfloat16 or float32 each; H is a multiple
    of 8 up to 16384.  h is the float32 sum in the residual's type, kept in residual_out (new
    memory, the residual itself, or x itself where type and strides are the same) and
    normalised as kept.  dtype torch.float8_e4m3fn (H a multiple of 128) gives codes with
    their scales per 128 columns, as source_dispatch takes them: scale = amax / 448 of the
    float32 y, 0 below 2^-126.  x, residual and residual_out may have gaps between rows
    (16-byte aligned, strides in multiples of 8); out is contiguous, and may be a bfloat16 x.
    keep_rstd: also 1 / sqrt(mean(h^2) + eps), for rms_norm_grad.

    Differentiable by x, residual and weight with bfloat16 rows in new memory, outside of
    a capture; the rounding of h counts as none, and x and residual share one gradient.
    Runs on x's device and its current stream."""
    eps = float(eps)
    given = out is not None or out_scales is not None or residual_out is not None
    if given:
        _plain("rms_norm", out, out_scales, residual_out)
    if _asks(x, weight, residual):
        _recorded("rms_norm", x.device, out is not None, out_scales is not None, residual_out is not None,
                  dtype is not torch.bfloat16)
        rows, h, rstd = _RmsNorm.apply(x, weight, residual, eps)
        return Normed(rows, None, h, rstd if keep_rstd else None)
    n = _norm(x, weight, residual, eps, dtype, out, out_scales, residual_out, keep_rstd)
    if given:
        wrote(out, out_scales, residual_out)
    return n


def rms_norm_grad(grad, h, weight, rstd, *, grad_residual=None, out=None, weight_grad=True):
    """The gradients (dh, dweight) of rms_norm with bfloat16 rows.

    grad bfloat16 [T, H], of the rows; h as rms_norm kept it (or x, without a residual), and
    its rstd; grad_residual: of h as the stream goes on, contiguous in h's type.  dh, in h's
    type, is the gradient of x and of the residual alike; out may be grad_residual, or a
    grad of h's type.  dweight is float32 [H], None without weight_grad."""
    _plain("rms_norm_grad", grad, h, weight, rstd, grad_residual, out)
    key = (h.dtype, h.shape, h.stride(), h.device, weight.dtype, weight.shape, weight.stride(), weight.device,
           _layout(grad), None if grad_residual is None else _layout(grad_residual), _layout(rstd),
           None if out is None else _layout(out))
    plan = _norm_grads.get(key) or _keep(_norm_grads, key, _norm_grad_plan(grad, h, weight, rstd, grad_residual, out))
    cfg, hs, need = plan
    (T, H), dev = h.shape, h.device
    given = out
    if out is None:
        out = _like(h, h.dtype)
    dw = ws = pd = pw = None
    if weight_grad:
        dw = torch.empty(H, dtype=torch.float32, device=dev)
        pd = dw.data_ptr()
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            pw = ws.data_ptr()
    st = _launch(dev, nat.load().afd_norm_grad, cfg, T, grad.data_ptr(),
                 None if grad_residual is None else grad_residual.data_ptr(), h.data_ptr(), hs, weight.data_ptr(),
                 rstd.data_ptr(), out.data_ptr(), pd, pw, need if weight_grad else 0)
    if st:
        _check(st, "rms_norm_grad", grad=grad, grad_residual=grad_residual, h=h, weight=weight, out=out)
    if given is not None:
        wrote(given)
    return out, dw


def _norm_grad_plan(grad, h, weight, rstd, grad_residual, out):
    """(configuration, row stride of h, workspace bytes) of a norm's gradient whose arguments' layouts fit."""
    hs = _wide_rows(h, "h")
    (T, H), dev = h.shape, h.device
    _want(weight, "weight", weight.dtype, (H,), dev)
    _want(grad, "grad", torch.bfloat16, (T, H), dev)
    if grad_residual is not None:
        _want(grad_residual, "grad_residual", h.dtype, (T, H), dev)
    _want(rstd, "rstd", torch.float32, (T,), dev)
    if out is not None:
        _want(out, "out", h.dtype, (T, H), dev)
    cfg, ws = _norm_config(H, _code(h, "h"), nat.NO_RESIDUAL, _code(weight, "weight"), nat.AFD_BF16, 1.0), ctypes.c_size_t(0)
    nat.check(nat.load().afd_norm_grad_query(ctypes.byref(cfg), T, ctypes.byref(ws)), "rms_norm_grad")
    return cfg, hs, ws.value


@functools.lru_cache(maxsize=256)
def _route_config(experts, topk, code, scoring, renormalize, scale):
    if not 0 < experts <= nat.MAX_EXPERTS:
        raise ValueError(f"logits must have 1 to {nat.MAX_EXPERTS} experts, got {experts}")
    if not 0 < topk <= min(nat.MAX_TOPK, experts):
        raise ValueError(f"topk must be 1 to {min(nat.MAX_TOPK, experts)} of {experts} experts, got {topk}")
    if scoring not in nat.SCORINGS:
        raise ValueError(f"scoring must be one of {sorted(nat.SCORINGS)}, got {scoring!r}")
    if not abs(scale) <= torch.finfo(torch.float32).max:
        raise ValueError(f"scale must be a finite float32, got {scale}")
    return nat.RouteConfig(experts, topk, code, nat.SCORINGS[scoring], int(renormalize), scale)


def _ids_of(ids, logits):
    """ids [T, topk] beside the logits."""
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, topk], got {list(ids.shape)}")
    _want(ids, "ids", torch.int32, (logits.shape[0], ids.shape[1]), logits.device)
    return ids.shape[1]


def _route_plan(logits, topk, scoring, bias, renormalize, scale, live, ids, weights):
    """(configuration, row stride) of a choice whose arguments' layouts fit."""
    ls = _rows(logits, "logits")
    (T, E), dev = logits.shape, logits.device
    cfg = _route_config(E, topk, _code(logits, "logits"), scoring, renormalize, scale)
    if bias is not None:
        _want(bias, "bias", torch.float32, (E,), dev)
    if live is not None:
        _want(live, "live", torch.bool, (T,), dev)
    if ids is not None:
        _want(ids, "ids", torch.int32, (T, cfg.topk), dev)
    if weights is not None:
        _want(weights, "weights", torch.float32, (T, cfg.topk), dev)
    return cfg, ls


def _route(logits, topk, scoring, bias, renormalize, scale, live, ids, weights):
    key = (logits.dtype, logits.shape, logits.stride(), logits.device, topk, scoring, renormalize, scale,
           None if bias is None else _layout(bias), None if live is None else _layout(live),
           None if ids is None else _layout(ids), None if weights is None else _layout(weights))
    plan = _routes.get(key) or _keep(_routes, key, _route_plan(logits, topk, scoring, bias, renormalize, scale, live, ids,
                                                               weights))
    cfg, ls = plan
    T, dev = logits.shape[0], logits.device
    if ids is None:
        ids = torch.empty((T, cfg.topk), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty_like(ids, dtype=torch.float32)
    st = _launch(dev, nat.load().afd_route, cfg, T, logits.data_ptr(), ls, None if bias is None else bias.data_ptr(),
                 None if live is None else live.data_ptr(), ids.data_ptr(), weights.data_ptr())
    if st:
        nat.check(st, "route_tokens")
    return Routes(ids, weights)


class _RouteTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, scoring, bias, renormalize, scale, live):
        r = _route(logits, topk, scoring, bias, renormalize, scale, live, None, None)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(r.ids)
        ctx.save_for_backward(logits, r.ids)
        ctx.how = dict(scoring=scoring, renormalize=renormalize, scale=scale)
        return r.ids, r.weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, grad):
        if grad is None:
            return (None,) * 7
        logits, ids = ctx.saved_tensors
        with on_device(logits.device):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("route_tokens: its backward pass is not captured: call route_tokens_grad")
        return (route_tokens_grad(grad.contiguous(), logits, ids, **ctx.how),) + (None,) * 6


def route_tokens(logits, topk, *, scoring="softmax", bias=None, renormalize=True, scale=1.0, live=None, ids=None,
                 weights=None) -> Routes:
    """Every token's topk experts and their weights, as source_dispatch takes them.

    logits [T, E] bfloat16 or float32, E up to 512, topk up to 32; rows may have gaps.
    Scores are the logits' "softmax" or "sigmoid".  ids are in falling order of score, with
    bias (float32 [E]) of score + bias, the lower id first where equal (compared as 64-bit
    scores with a bias, as logits without).  weights are scale * score, with renormalize
    divided by the sum of the token's chosen scores; the bias is not in them.  live (bool
    [T]): tokens that are False have ids -1 and weights 0.  An expert whose logit (or score
    + bias) is minus infinity or NaN is never chosen; ids that are left over are -1, with
    weight 0.  Weights are within 32 float32 roundings (2^-24 each) of their definition.  ids and
    weights: memory for the results.

    The weights are differentiable by the logits, outside of a capture; the choice has no
    gradient.  Runs on the logits' device and its current stream."""
    topk, renormalize, scale = operator.index(topk), bool(renormalize), float(scale)
    if bias is not None or live is not None or ids is not None or weights is not None:
        _plain("route_tokens", bias, live, ids, weights)
    if _asks(logits):
        _recorded("route_tokens", logits.device, ids is not None, weights is not None)
        return Routes(*_RouteTokens.apply(logits, topk, scoring, bias, renormalize, scale, live))
    r = _route(logits, topk, scoring, bias, renormalize, scale, live, ids, weights)
    if ids is not None or weights is not None:
        wrote(ids, weights)
    return r


def route_tokens_grad(grad, logits, ids, *, scoring="softmax", renormalize=True, scale=1.0, out=None):
    """The logits' gradient, [T, E] of their type, through the weights of route_tokens: grad float32
    [T, topk], ids as they were chosen (any outside [0, E) takes no part)."""
    renormalize, scale = bool(renormalize), float(scale)
    _plain("route_tokens_grad", grad, logits, ids, out)
    grad = grad.resolve_neg()       # autograd may hold back a sign, which the memory then lacks
    key = (logits.dtype, logits.shape, logits.stride(), logits.device, scoring, renormalize, scale, _layout(grad), _layout(ids),
           None if out is None else _layout(out))
    plan = _routes.get(key) or _keep(_routes, key, _route_grad_plan(grad, logits, ids, scoring, renormalize, scale, out))
    cfg, ls = plan
    given = out
    if out is None:
        out = _like(logits, logits.dtype)
    st = _launch(logits.device, nat.load().afd_route_grad, cfg, logits.shape[0], grad.data_ptr(), logits.data_ptr(), ls,
                 ids.data_ptr(), out.data_ptr())
    if st:
        nat.check(st, "route_tokens_grad")
    if given is not None:
        wrote(given)
    return out


def _route_grad_plan(grad, logits, ids, scoring, renormalize, scale, out):
    ls, topk = _rows(logits, "logits"), _ids_of(ids, logits)
    _want(grad, "grad", torch.float32, tuple(ids.shape), logits.device)
    if out is not None:
        _want(out, "out", logits.dtype, tuple(logits.shape), logits.device)
    return _route_config(logits.shape[1], topk, _code(logits, "logits"), scoring, renormalize, scale), ls


def _balance_plan(logits, ids, scoring, coefficient):
    """(configuration, row stride, workspace bytes) of a loss whose arguments' layouts fit."""
    ls, topk = _rows(logits, "logits"), _ids_of(ids, logits)
    cfg, ws = _route_config(logits.shape[1], topk, _code(logits, "logits"), scoring, False, 1.0), ctypes.c_size_t(0)
    if not abs(coefficient) <= torch.finfo(torch.float32).max:
        raise ValueError(f"coefficient must be a finite float32, got {coefficient}")
    nat.check(nat.load().afd_balance_query(ctypes.byref(cfg), logits.shape[0], ctypes.byref(ws)), "balance_loss")
    return cfg, ls, ws.value


def _balance(logits, ids, scoring, coefficient):
    key = logits.dtype, logits.shape, logits.stride(), logits.device, _layout(ids), scoring, coefficient
    plan = _balances.get(key) or _keep(_balances, key, _balance_plan(logits, ids, scoring, coefficient))
    cfg, ls, need = plan
    (T, E), dev = logits.shape, logits.device
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    slope = torch.empty_like(counts, dtype=torch.float32)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = _launch(dev, nat.load().afd_balance, cfg, T, logits.data_ptr(), ls, ids.data_ptr(), coefficient, loss.data_ptr(),
                 counts.data_ptr(), slope.data_ptr(), ws.data_ptr() if need else None, need)
    if st:
        nat.check(st, "balance_loss")
    return Balance(loss, counts, slope)


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, scoring, coefficient):
        b = _balance(logits, ids, scoring, coefficient)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(b.counts, b.slope)
        ctx.save_for_backward(logits, ids, b.slope)
        ctx.scoring = scoring
        return tuple(b)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, *_):
        if grad is None:
            return None, None, None, None
        logits, ids, slope = ctx.saved_tensors
        with on_device(logits.device):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("balance_loss: its backward pass is not captured: call balance_loss_grad")
        return balance_loss_grad(grad, logits, ids, slope, scoring=ctx.scoring), None, None, None


def balance_loss(logits, ids, *, scoring="softmax", coefficient=1.0) -> Balance:
    """The experts' loads and the loss that keeps them even, of the tokens that have an expert.

    logits [T, E] as in route_tokens, ids int32 [T, topk] (route_tokens' or any; those
    outside [0, E) are skipped, and a token with no other does not count).  With n counting
    tokens, C choices in all and share[t, e] a token's softmax (or its sigmoids, divided by
    their sum): slope[e] = coefficient * E * counts[e] / (C * n) and loss = sum of slope[e] *
    share[t, e] over counting tokens and experts, which is the coefficient where use and
    shares are even.  Without a counting token the loss is 0.

    The loss is differentiable by the logits, through the shares, outside of a capture.
    Runs on the logits' device and its current stream."""
    coefficient = float(coefficient)
    _plain("balance_loss", ids)
    if _asks(logits):
        _recorded("balance_loss", logits.device)
        return Balance(*_BalanceLoss.apply(logits, ids, scoring, coefficient))
    return _balance(logits, ids, scoring, coefficient)


def balance_loss_grad(grad, logits, ids, slope, *, scoring="softmax", out=None):
    """The logits' gradient, [T, E] of their type: grad float32 [], of the loss on the GPU;
    ids and slope as balance_loss had and gave them.  Tokens that do not count have 0."""
    _plain("balance_loss_grad", grad, logits, ids, slope, out)
    grad = grad.resolve_neg()
    key = (logits.dtype, logits.shape, logits.stride(), logits.device, _layout(ids), scoring, _layout(grad), _layout(slope),
           None if out is None else _layout(out))
    plan = _balances.get(key) or _keep(_balances, key, _balance_grad_plan(grad, logits, ids, slope, scoring, out))
    cfg, ls = plan
    given = out
    if out is None:
        out = _like(logits, logits.dtype)
    st = _launch(logits.device, nat.load().afd_balance_grad, cfg, logits.shape[0], grad.data_ptr(), logits.data_ptr(), ls,
                 ids.data_ptr(), slope.data_ptr(), out.data_ptr())
    if st:
        nat.check(st, "balance_loss_grad")
    if given is not None:
        wrote(given)
    return out


def _balance_grad_plan(grad, logits, ids, slope, scoring, out):
    ls, topk = _rows(logits, "logits"), _ids_of(ids, logits)
    _want(grad, "grad", torch.float32, (), logits.device)
    _want(slope, "slope", torch.float32, (logits.shape[1],), logits.device)
    if out is not None:
        _want(out, "out", logits.dtype, tuple(logits.shape), logits.device)
    return _route_config(logits.shape[1], topk, _code(logits, "logits"), scoring, False, 1.0), ls
