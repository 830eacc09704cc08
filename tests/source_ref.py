"""The source's side in 64 bits on the CPU, with bounds that count roundings.

U is half a float32 step.  A float32 sum of n terms in any order is off by at
most n * U times the sum of their sizes (to first order; the slack of the counts
below covers the rest).
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126            # below it float32 results may be 0
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U, torch.float8_e4m3fn: 2.0 ** -4}
INF = float("inf")


def adds(hidden):
    """Float32 additions that a term of a row's sum meets: at most eight runs of eight in a
    lane, six steps across a wavefront and one for each of 16 wavefronts."""
    return 64 + 6 + 16


def norm(x, weight, residual, eps):
    """(h as stored, rstd, y) and the relative bound of rstd (float64, CPU)."""
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(residual.dtype).double()     # defined as the float32 sum
    ms = h.square().mean(1)
    rstd = 1 / torch.sqrt(ms + eps)
    # each square is rounded once inside a fused addition; the division, the addition of
    # eps and the root's one step (2 U) follow, and a root halves what comes before it
    rel = (adds(h.shape[1]) + 4) * U / 2 + 3 * U
    return h, rstd, h * rstd[:, None] * weight.double(), rel


def norm_grad(grad, h, weight, rstd, grad_residual):
    """(dh, its bound, dweight, its bound) of float64 inputs."""
    H = h.shape[1]
    u, a = h * rstd[:, None], grad * weight
    m = (a * u).mean(1, keepdim=True)
    dh = rstd[:, None] * (a - u * m)
    # a and u are rounded once each, their product inside the addition; m once more by the division
    dm = ((adds(H) + 4) * U) * (a * u).abs().mean(1, keepdim=True)
    tol = rstd[:, None] * (4 * U * a.abs() + u.abs() * (dm + 4 * U * m.abs()))
    if grad_residual is not None:
        dh = dh + grad_residual
    tol = tol + 3 * U * dh.abs()
    rows = grad.shape[0]
    # up to 1024 rows: every 32nd row in a thread, then 32 threads (128th and 128 where wide); more: a
    # workgroup's rows (of up to 512) one after another, four wavefronts, every 64th workgroup, then 64 sums
    terms = rows / 32 + 1 + 128 if rows <= 1024 else rows / min(-(-rows // 4), 512) + 1 + 4 + 512 / 64 + 64
    return dh, tol, (grad * u).sum(0), (terms + 3) * U * (grad * u).abs().sum(0)


def clean(logits):
    v = logits.double()
    return torch.where(v.isnan(), -INF, v)


def scores(logits, scoring):
    """Scores by definition; experts at plus infinity share a softmax."""
    v = clean(logits)
    if scoring == "sigmoid":
        return torch.sigmoid(v)
    m = v.amax(1, keepdim=True)
    t = torch.where(v == -INF, 0.0, torch.where(v == m, 1.0, torch.exp(v - m)))
    s = t.sum(1, keepdim=True)
    return t / torch.where(s > 0, s, 1.0)


def log_scores(logits, scoring):
    """Their logarithms but for a factor common to the row, which no range hides."""
    v = clean(logits)
    if scoring == "softmax":
        return v
    return torch.where(v == -INF, -INF, -torch.nn.functional.softplus(-v))


def choose(logits, topk, scoring, bias, live):
    key = clean(logits)
    if bias is not None:
        x = scores(logits, scoring) + bias.double()
        key = torch.where((key == -INF) | x.isnan(), -INF, x)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = torch.where(top[:, :topk] == -INF, -1, ids[:, :topk])
    if live is not None:
        ids = torch.where(live[:, None], ids, -1)
    return ids


def spread(logits):
    """Roundings of an exponential's argument and of the sums around it, in U: the argument
    is a difference of up to 120 (below, the term is 0), rounded once."""
    v = clean(logits)
    m = v.amax(1, keepdim=True)
    d = torch.where(v == -INF, 0.0, m - v).nan_to_num(0.0, 120.0, 0.0).clamp(max=120.0).amax(1, keepdim=True)
    return 2 * d + 64


def weights(logits, ids, scoring, renormalize, scale):
    """Weights [T, K] in float64 and their bound."""
    on, at = ids >= 0, ids.clamp(min=0)
    if renormalize:
        l = torch.where(on, torch.take_along_dim(log_scores(logits, scoring), at, 1), -INF)
        m = l.amax(1, keepdim=True)
        t = torch.where(l == -INF, 0.0, torch.where(l == m, 1.0, torch.exp(l - m)))
        s = t.sum(1, keepdim=True)
        w = t / torch.where(s > 0, s, 1.0)
    else:
        w = torch.where(on, torch.take_along_dim(scores(logits, scoring), at, 1), 0.0)
    w = scale * w
    return w, spread(logits) * U * w.abs() + TINY * abs(scale)


def route_grad(grad, logits, ids, scoring, renormalize, scale):
    """dlogits [T, E] in float64 and its bound."""
    on = (ids >= 0) & (ids < logits.shape[1])
    at = torch.where(on, ids, 0)
    g = torch.where(on, grad.double(), 0.0) * scale
    v = clean(logits)
    w = weights(logits, torch.where(on, ids, -1), scoring, renormalize, 1.0)[0]
    left = torch.sigmoid(-torch.take_along_dim(v, at, 1)) if scoring == "sigmoid" else torch.ones_like(w)
    dot, size = (g * w).sum(1, keepdim=True), (g * w).abs().sum(1, keepdim=True)
    base = dot if renormalize else torch.zeros_like(dot)
    c = torch.where(on, w * left * (g - base), 0.0)
    ct = torch.where(on, w * left * (g.abs() + (size if renormalize else 0.0)), 0.0)
    d = torch.zeros_like(v).scatter_add(1, at, c)
    t = torch.zeros_like(v).scatter_add(1, at, ct)
    if scoring == "softmax" and not renormalize:
        p = scores(logits, scoring)
        d, t = d - p * dot, t + p * size
    k = ids.shape[1]
    return d, 3 * (spread(logits) + k) * U * t + 4 * TINY * (1 + g.abs().amax(1, keepdim=True))


def shares(logits, scoring):
    l = log_scores(logits, scoring)
    m = l.amax(1, keepdim=True)
    t = torch.where(l == -INF, 0.0, torch.where(l == m, 1.0, torch.exp(l - m)))
    s = t.sum(1, keepdim=True)
    return t / torch.where(s > 0, s, 1.0)


def balance(logits, ids, scoring, coefficient):
    """loss and its bound, counts, slope, shares of the counting tokens, the counting tokens."""
    E = logits.shape[1]
    ok = (ids >= 0) & (ids < E)
    on = ok.any(1)
    counts = torch.bincount(ids[ok].long(), minlength=E)
    n = int(on.sum()) * int(counts.sum())
    slope = coefficient * E * counts.double() / n if n else torch.zeros(E, dtype=torch.float64)
    p = shares(logits, scoring) * on[:, None]
    loss = (p.sum(0) * slope).sum()
    rows = p.shape[0]
    # a lane's tokens one after another, then up to 64 groups of a workgroup; the join is in 64 bits
    terms = rows / 256 + 6 + 64
    worst = float((spread(logits)).max()) if rows else 0.0
    return loss, (terms + worst + 4) * U * (p.sum(0) * slope.abs()).sum() + TINY, counts, slope, p, on


def balance_grad(grad, logits, p, slope, on, scoring):
    v = clean(logits)
    left = torch.sigmoid(-v) if scoring == "sigmoid" else torch.ones_like(v)
    dot, size = (p * slope).sum(1, keepdim=True), (p * slope.abs()).sum(1, keepdim=True)
    d = grad * p * left * (slope - dot)
    t = abs(grad) * p * left * (slope.abs() + size)
    return torch.where(on[:, None], d, 0.0), 3 * spread(logits) * U * t + 4 * TINY * (1 + abs(grad) * size)


def rounded(want, tol, dtype):
    """The bound behind one rounding to dtype."""
    sub = 2.0 ** -134 if dtype is torch.bfloat16 else 2.0 ** -150
    return tol + HALF_STEP[dtype] * (want.abs() + tol) + sub


def check(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    err = (got - want).abs()
    bad = ~((err <= tol) | (got == want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((err / tol).nan_to_num(INF).max())} of the bound")
