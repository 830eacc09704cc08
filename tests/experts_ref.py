"""Plain 64-bit reference of the experts' side on the CPU, with bounds on how
far a right result can be from it.

The bounds count roundings: float32 sums of n terms are off by at most
n * 2^-24 * sum |terms| (each addition or multiply by 2^-24 of what it holds,
whatever the order), a BF16 rounding by 2^-8 of the value, an E4M3 rounding by
2^-4 of the value or, below the smallest normal number 2^-6, by 2^-10 steps of
the block's scale.
"""
import numpy as np
import torch

F32, BF16 = 2.0 ** -24, 2.0 ** -8
RATE = 448.0


def spans(ends, alpha, rows):
    """[first, last) of every expert, cut at `rows`."""
    out, prev = [], 0
    for e in ends:
        s = -(-min(max(prev, 0), rows) // alpha) * alpha
        out.append((s, max(min(int(e), rows), s)) if s <= rows else (rows, rows))
        prev = int(e)
    return out


def layout(counts, alpha):
    ends, at = [], 0
    for c in counts:
        at = -(-at // alpha) * alpha + c
        ends.append(at)
    return ends


def quant(v, block_rows):
    """E4M3 codes and float32 scales per block_rows x 128 of v [..., n, k]."""
    n, k = v.shape[-2:]
    nb = -(-n // block_rows)
    pad = torch.zeros(*v.shape[:-2], nb * block_rows, k)
    pad[..., :n, :] = v
    s = (pad.abs().reshape(*v.shape[:-2], nb, block_rows, k // 128, 128).amax((-3, -1)) / RATE).float()
    full = s.repeat_interleave(block_rows, -2)[..., :n, :].repeat_interleave(128, -1)
    return (v / torch.where(full > 0, full, torch.ones(()))).to(torch.float8_e4m3fn), s


def wide(q, s, block_rows=1):
    v = q.double()
    if s is None:
        return v
    return v * s.double().repeat_interleave(block_rows, -2)[..., :v.shape[-2], :].repeat_interleave(128, -1)


def silu(g):
    return g * torch.sigmoid(g)


def product(x, dx, w, gated, low, tags, j):
    """Values and error bound (before the output's rounding) of act(x w^T)
    for x [r, k] known within dx; low = (a [S, E, c*r, k], b, scaling)."""
    n = x.shape[1]
    xa, wa = x.abs() + dx, w.abs()
    # + 2 roundings per scaled block of an FP8 sum, counted with the terms
    y, dy = x @ w.t(), dx @ wa.t() + (n + 4) * F32 * (xa @ wa.t())
    if low is not None:
        a, b, sc = (t.double() for t in low)
        S, rank = sc.shape[0], b.shape[-1]
        for i in range(S):
            at = (tags == i).nonzero().reshape(-1)
            if len(at) == 0:
                continue
            half = w.shape[0] // 2
            for c in range(2 if gated else 1):
                cols = slice(c * half, (c + 1) * half) if gated else slice(0, w.shape[0])
                A, B = a[i, j, c * rank:(c + 1) * rank], b[i, j, cols]
                t = sc[i] * (x[at] @ A.t())
                # t in float32 and in two bf16 parts (off by 2^-17 of t)
                dt = sc[i].abs() * (dx[at] @ A.abs().t() + (n + 4) * F32 * (xa[at] @ A.abs().t())) + 2.0 ** -16 * t.abs()
                y[at, cols] += t @ B.t()
                dy[at, cols] += dt @ B.abs().t() + (rank + 4) * F32 * ((t.abs() + dt) @ B.abs().t())
        dy += 4 * F32 * (y.abs() + dy)
    if not gated:
        return y, dy
    g, u = y.chunk(2, 1)
    dg, du = dy.chunk(2, 1)
    h = silu(g) * u
    # |silu'| <= 1.1; exp, division and product off by a few float32 steps, and
    # exp's argument rounding by 2^-24 |g| of the exponential
    dh = 1.1 * dg * (u.abs() + du) + (silu(g).abs() + 1.1 * dg) * du + (16 + 2 * g.abs()) * F32 * h.abs()
    return h, dh


def run_product(case, x, xs, w, ws, low, tags, ends, alpha, rows):
    """float64 result [rows, n] and bound (before rounding), live-row mask."""
    gated = case["gated"]
    n = w.shape[1] // (2 if gated else 1)
    out, tol = torch.zeros(rows, n, dtype=torch.float64), torch.zeros(rows, n, dtype=torch.float64)
    live = torch.zeros(rows, dtype=torch.bool)
    for j, (s, e) in enumerate(spans(ends, alpha, rows)):
        if s >= e:
            continue
        v = wide(x[s:e], None if xs is None else xs[s:e])
        out[s:e], tol[s:e] = product(v, torch.zeros_like(v), wide(w[j], None if ws is None else ws[j], 128), gated, low,
                                     None if tags is None else tags[s:e], j)
        live[s:e] = True
    return out, tol, live


def run_ffn(x, xs, up, ups, down, downs, lu, ld, tags, ends, alpha, rows):
    out = torch.zeros(rows, down.shape[1], dtype=torch.float64)
    tol = torch.zeros_like(out)
    live = torch.zeros(rows, dtype=torch.bool)
    for j, (s, e) in enumerate(spans(ends, alpha, rows)):
        if s >= e:
            continue
        t = None if tags is None else tags[s:e]
        v = wide(x[s:e], None if xs is None else xs[s:e])
        h, dh = product(v, torch.zeros_like(v), wide(up[j], None if ups is None else ups[j], 128), True, lu, t, j)
        if xs is None:
            dh = dh + BF16 * (h.abs() + dh)
        else:
            m = (h.abs() + dh).reshape(e - s, -1, 128).amax(-1) / RATE
            dh = dh + 2.0 ** -4 * (h.abs() + dh) + (2.0 ** -10 * m).repeat_interleave(128, 1)
        out[s:e], tol[s:e] = product(h, dh, wide(down[j], None if downs is None else downs[j], 128), False, ld, t, j)
        live[s:e] = True
    return out, tol, live


def rounded(out, tol):
    """The bound after one BF16 rounding (and its subnormal step)."""
    return tol + BF16 * (out.abs() + tol) + 2.0 ** -134


def make(seed, E, counts, alpha, k, m, dtype, S=0, rank=0, gated=False, extra_rows=3):
    """Inputs on the CPU; padding rows of x hold NaN (bf16) or NaN codes."""
    g = torch.Generator().manual_seed(seed)
    ends = layout(counts, alpha)
    rows = (ends[-1] if ends else 0) + extra_rows
    x = torch.randn(rows, k, generator=g)
    w = torch.randn(E, m, k, generator=g) * k ** -0.5
    live = torch.zeros(rows, dtype=torch.bool)
    for s, e in spans(ends, alpha, rows):
        live[s:e] = True
    if dtype == "fp8":
        xq, xs = quant(x, 1)
        wq, ws = quant(w, 128)
        xq.view(torch.uint8)[~live] = 0x7F
        xs[~live] = float("nan")
    else:
        xq, xs, wq, ws = x.bfloat16(), None, w.bfloat16(), None
        xq[~live] = float("nan")
    low = tags = None
    if S:
        c = 2 if gated else 1
        low = ((torch.randn(S, E, c * rank, k, generator=g) * k ** -0.5).bfloat16(),
               (torch.randn(S, E, m, rank, generator=g) * rank ** -0.5).bfloat16(),
               torch.rand(S, generator=g) + 0.25)
        # runs and single rows, some without an adapter, some out of range
        tags = torch.randint(-1, S, (rows,), generator=g, dtype=torch.int32)
        tags[torch.rand(rows, generator=g) < 0.1] = S
        tags[torch.rand(rows, generator=g) < 0.05] = -(2 ** 31)
        half = rows // 2
        tags[half:] = tags[half:][torch.arange(rows - half) // 7 * 7]
    return dict(x=xq, xs=xs, w=wq, ws=ws, low=low, tags=tags, ends=ends, rows=rows, live=live, alpha=alpha, gated=gated)


def as_np(t):
    return t.numpy() if isinstance(t, torch.Tensor) else np.asarray(t)
