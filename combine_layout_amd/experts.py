"""Python binding of the experts' side of a round: products grouped by expert,
the experts' network, and low-rank adapters beside their projections.

Argument checks and marshalling only: the arithmetic runs in the HIP library.
Rows are laid out as ``Buffer.worker_receive`` hands them out: expert j owns
rows [align_up(ends[j-1], alignment), ends[j]).  Rows inside no expert's range
are neither read nor written.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _native as nat

SCALE_BLOCK = 128


class LowRank(NamedTuple):
    """One projection's adapters: scaling[i] * B_ij (A_ij x) beside expert j's.
    For a gated projection A holds the gate's rank rows, then the up's."""
    a: torch.Tensor        # [S, E, rank or 2*rank, k] bf16
    b: torch.Tensor        # [S, E, rows of the weight, rank] bf16
    scaling: torch.Tensor  # [S] float32


class PackedWeights:
    """Weights [E, m, k] in the order in which the products read them (made by
    pack_weights); takes the place of the row-major tensor in the calls."""

    def __init__(self, data, shape, dtype):
        self.data, self.shape, self.dtype, self.device = data, torch.Size(shape), dtype, data.device


def pack_weights(w) -> PackedWeights:
    """A packed copy of row-major weights [E, m, k], bf16 or float8_e4m3fn, m a
    multiple of 16 and k of 64 (float8: 128).  The products read runs of
    1024 bytes of it, faster than rows; the results are the same.  The copy has no
    gradient: weights that ask for one are refused unless gradients are off."""
    if isinstance(w, PackedWeights):
        return w
    _no_gradients(w)
    if w.dim() != 3 or w.device.type != "cuda" or not w.is_contiguous():
        raise ValueError("weights must be a contiguous [E, m, k] tensor on a GPU")
    E, m, k = w.shape
    code, _ = _act_dtype(w)
    c = _config(nat.ProductConfig, E, 1, k, m, code, nat.AFD_BF16, nat.AFD_ACT_NONE, 0, 0, nat.WEIGHTS_ROWS)
    data = torch.empty(w.numel() * w.element_size(), dtype=torch.uint8, device=w.device)
    with on_device(w.device):
        st = nat.load().afd_pack_weights(c, w.data_ptr(), data.data_ptr(), raw_stream(w.device))
    nat.check(st, "pack_weights")
    return PackedWeights(data, w.shape, w.dtype)


class Experts:
    """Weights of a partition's experts, bf16, or float8_e4m3fn with float32
    scales per 128 x 128 block, laid out once: up and down are kept as packed
    copies (pack_weights), and the tensors passed here can go.  Like the copies,
    the scales are kept without a gradient, and refused where they ask for one.

    up [E, 2*inner, hidden] (gate rows, then up rows), down [E, hidden, inner],
    up_scales [E, 2*inner/128, hidden/128], down_scales [E, hidden/128, inner/128]."""

    def __init__(self, up, down, up_scales=None, down_scales=None):
        _no_gradients(up_scales, down_scales)
        self.up, self.down = pack_weights(up), pack_weights(down)
        self.up_scales, self.down_scales = (None if s is None else s.detach() for s in (up_scales, down_scales))


class ExpertAdapters(NamedTuple):
    up: LowRank
    down: LowRank


_SAME_DEVICE = contextlib.nullcontext()


def on_device(device):
    """The current device for a launch, changed only where it differs."""
    return _SAME_DEVICE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def raw_stream(device):
    """The device's current stream as a hipStream_t, without the Stream object
    that torch.cuda.current_stream makes (about 2 us of a call's 10)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def wrote(*given):
    """The kernels write by address, which autograd does not see: a graph that saved one of the
    given outputs has to find it changed.  (Tensors of inference mode have no counter.)"""
    increment_version([t for t in given if t is not None])


def _config(kind, *values):
    """The configuration of int32 values; what no int32 holds is refused, not cut."""
    for (name, _), v in zip(kind._fields_, values):
        if not (name == "alignment") <= v < 2 ** 31:
            raise ValueError(f"{name} must be in [{int(name == 'alignment')}, 2^31), got {v}")
    return kind(*values)


@functools.lru_cache(maxsize=256)
def _product_plan(rows, *cfg):
    c, ws = _config(nat.ProductConfig, *cfg), ctypes.c_size_t(0)
    nat.check(nat.load().afd_product_query(ctypes.byref(c), rows, ctypes.byref(ws)), "expert_product")
    return c, ws.value


@functools.lru_cache(maxsize=256)
def _ffn_plan(rows, *cfg):
    c, ws = _config(nat.FfnConfig, *cfg), ctypes.c_size_t(0)
    nat.check(nat.load().afd_ffn_query(ctypes.byref(c), rows, ctypes.byref(ws)), "expert_ffn")
    return c, ws.value


def _want(t, what, dtype, shape, device):
    if t is None or t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on {device}, got " + (
            "None" if t is None else f"{t.dtype} {list(t.shape)} on {t.device}, contiguous {t.is_contiguous()}"))
    return t.data_ptr()


def _act_dtype(x):
    """(dtype code, torch dtype) of activations and weights."""
    if x.dtype is torch.bfloat16:
        return nat.AFD_BF16, torch.bfloat16
    if x.dtype is torch.float8_e4m3fn:
        return nat.AFD_FP8_E4M3, torch.float8_e4m3fn
    raise TypeError("x must be bfloat16 or float8_e4m3fn")


def _number_and_rank(low):
    if low.scaling.dim() != 1 or low.b.dim() != 4:
        raise ValueError("adapters hold a [S, E, rank or 2*rank, k], b [S, E, m, rank] and scaling [S]")
    return low.scaling.shape[0], low.b.shape[3]


def _no_gradients(*tensors):
    """These are forward calls: what asks for a gradient, or carries a forward
    one, would silently lose it."""
    if torch.is_grad_enabled():
        for t in tensors:
            if getattr(t, "requires_grad", False):
                raise ValueError("the experts' calls have no gradients: detach their inputs or call under no_grad()")
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("the experts' calls have no gradients: pass the primal of a dual tensor")


def _weights(what, w, scales, low, E, m, k, code, dtype, gated, device):
    """The checked pointers of one product's weights."""
    p = nat.ProductWeights()
    if isinstance(w, PackedWeights):
        if w.dtype is not dtype or w.shape != (E, m, k) or w.device != device:
            raise ValueError(f"{what} weight must be {dtype} {[E, m, k]} on {device}, got {w.dtype} {list(w.shape)} on "
                             f"{w.device}")
        p.w = w.data.data_ptr()
    else:
        p.w = _want(w, f"{what} weight", dtype, (E, m, k), device)
    if code == nat.AFD_FP8_E4M3:
        p.w_scales = _want(scales, f"{what} weight scales", torch.float32, (E, -(-m // SCALE_BLOCK), k // SCALE_BLOCK),
                           device)
    elif scales is not None:
        raise ValueError("weight scales belong to float8_e4m3fn weights")
    if low is not None:
        S, rank = _number_and_rank(low)
        p.a = _want(low.a, f"{what} adapters' A", torch.bfloat16, (S, E, rank * (2 if gated else 1), k), device)
        p.b = _want(low.b, f"{what} adapters' B", torch.bfloat16, (S, E, m, rank), device)
        p.scaling = _want(low.scaling, f"{what} adapters' scaling", torch.float32, (S,), device)
    return p


def _rows(x, ends, x_scales, code, adapters, row_adapters, device):
    """The checked pointers of ends, the row scales and the rows' adapters."""
    R, k = x.shape
    pe = _want(ends, "ends", torch.int32, (ends.shape[0],), device)
    ps = pa = None
    if code == nat.AFD_FP8_E4M3:
        ps = _want(x_scales, "x_scales", torch.float32, (R, k // SCALE_BLOCK), device)
    elif x_scales is not None:
        raise ValueError("x_scales belong to float8_e4m3fn rows")
    if adapters is not None:
        pa = _want(row_adapters, "row_adapters", torch.int32, (R,), device)
    elif row_adapters is not None:
        raise ValueError("row_adapters without adapters")
    return pe, ps, pa


def _x(x):
    if x.dim() != 2 or not x.is_contiguous() or x.device.type != "cuda":
        raise ValueError("x must be a contiguous [rows, k] tensor on a GPU")
    return x.device


def expert_product(x, ends, weight, *, alignment=1, x_scales=None, weight_scales=None, activation=None, adapters=None,
                   row_adapters=None, out=None, out_scales=None, rows_per_expert=0):
    """out[r] = act(x[r] W_j^T) for the rows r of expert j, [rows, n] bf16.

    x [rows, k] bf16, or float8_e4m3fn with x_scales float32 [rows, k/128];
    weight [E, m, k] of the same type, or its pack_weights (float8:
    weight_scales float32 [E, ceil(m/128), k/128]); activation None (n = m) or "swiglu" (m = 2n, gate
    rows first).  k is a multiple of 64 (bf16) or 128, n of 16 (float8 swiglu:
    128).  adapters: a LowRank, with row_adapters int32 [rows] naming each
    row's (any value outside [0, S): none); rank a multiple of 8 up to 128.
    A float8 swiglu product writes float8 rows when `out` is a float8_e4m3fn
    tensor, with their scales in out_scales float32 [rows, n/128].
    Without `out` the result is new memory, its padding rows undefined.
    rows_per_expert: the rows that an expert is expected to have, by which a kernel
    is chosen (0: taken from the number of rows as worker_receive sizes them
    without host counts).
    Runs on x's device and its current stream; forward only (tensors that ask
    for a gradient are refused unless gradients are off, dual tensors always).
    """
    _no_gradients(x, weight, x_scales, weight_scales, out, out_scales, *(adapters or ()))
    dev = _x(x)
    R, k = x.shape
    code, dtype = _act_dtype(x)
    if activation not in nat.ACTIVATIONS:
        raise ValueError('activation must be None or "swiglu"')
    gated = activation == "swiglu"
    if len(weight.shape) != 3 or gated and weight.shape[1] % 2:
        raise ValueError("weight must be [E, m, k], m even with swiglu")
    E, m, _ = weight.shape
    n = m // 2 if gated else m
    if ends.dim() != 1 or ends.shape[0] != E:
        raise ValueError("ends must be int32 [E]")
    pe, ps, pa = _rows(x, ends, x_scales, code, adapters, row_adapters, dev)
    w = _weights("the", weight, weight_scales, adapters, E, m, k, code, dtype, gated, dev)
    out8 = out is not None and out.dtype is torch.float8_e4m3fn
    S, rank = _number_and_rank(adapters) if adapters is not None else (0, 0)
    cfg, need = _product_plan(R, E, alignment, k, n, code, nat.AFD_FP8_E4M3 if out8 else nat.AFD_BF16,
                              nat.ACTIVATIONS[activation], S, rank,
                              nat.WEIGHTS_PACKED if isinstance(weight, PackedWeights) else nat.WEIGHTS_ROWS,
                              rows_per_expert)
    given = out
    if out is None:
        out = torch.empty((R, n), dtype=torch.bfloat16, device=dev)
    po = _want(out, "out", torch.float8_e4m3fn if out8 else torch.bfloat16, (R, n), dev)
    pos = None
    if out8:
        pos = _want(out_scales, "out_scales", torch.float32, (R, n // SCALE_BLOCK), dev)
    elif out_scales is not None:
        raise ValueError("out_scales belong to a float8_e4m3fn out")
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    with on_device(dev):
        st = nat.load().afd_expert_product(cfg, R, x.data_ptr(), ps, pe, pa, w, po, pos,
                                           ws.data_ptr() if need else None, need,
                                           raw_stream(dev))
    nat.check(st, "expert_product")
    if given is not None:
        wrote(given, out_scales)
    return out


def expert_ffn(x, ends, experts: Experts, *, alignment=1, x_scales=None, adapters: Optional[ExpertAdapters] = None,
               row_adapters=None, out=None, rows_per_expert=0):
    """The experts' network, swiglu(x Wup^T) Wdown^T per expert, [rows, hidden]
    bf16.  Arguments as expert_product; the hidden layer is rounded to the
    rows' own format (bf16, or float8_e4m3fn with a scale per row and 128
    columns).  adapters: pairs beside both projections, of one rank and number.
    """
    _no_gradients(x, x_scales, out, *(adapters.up + adapters.down if adapters is not None else ()))
    dev = _x(x)
    R, hidden = x.shape
    code, dtype = _act_dtype(x)
    if experts.up.shape[1] % 2:
        raise ValueError("up must be [E, 2*inner, hidden]")
    E, inner = experts.up.shape[0], experts.up.shape[1] // 2
    if ends.dim() != 1 or ends.shape[0] != E:
        raise ValueError("ends must be int32 [E]")
    pe, ps, pa = _rows(x, ends, x_scales, code, adapters, row_adapters, dev)
    S = rank = 0
    if adapters is not None:
        S, rank = _number_and_rank(adapters.up)
        if _number_and_rank(adapters.down) != (S, rank):
            raise ValueError("both projections' adapters must have one number and rank")
    lu, ld = (adapters.up, adapters.down) if adapters is not None else (None, None)
    wu = _weights("up", experts.up, experts.up_scales, lu, E, 2 * inner, hidden, code, dtype, True, dev)
    wd = _weights("down", experts.down, experts.down_scales, ld, E, hidden, inner, code, dtype, False, dev)
    cfg, need = _ffn_plan(R, E, alignment, hidden, inner, code, S, rank, nat.WEIGHTS_PACKED, rows_per_expert)
    given = out
    if out is None:
        out = torch.empty((R, hidden), dtype=torch.bfloat16, device=dev)
    po = _want(out, "out", torch.bfloat16, (R, hidden), dev)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    with on_device(dev):
        st = nat.load().afd_expert_ffn(cfg, R, x.data_ptr(), ps, pe, pa, wu, wd, po, ws.data_ptr() if need else None, need,
                                       raw_stream(dev))
    nat.check(st, "expert_ffn")
    if given is not None:
        wrote(given)
    return out
