"""The source's side of a round as measurable cases: the norm that makes the
tokens a source dispatches (with the residual's addition, in BF16 or in E4M3
with block scales), the choice of every token's experts from its router's
logits, and the loss that keeps the experts evenly used; each with its
gradients where a router or a norm is trained.

``run`` computes a case in plain torch operations, or with ``own`` set through
the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK, LARGEST = 128, 448.0     # scale block, largest E4M3 value
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def _case(name, op, **kw):
    # tokens: per source.  norm: dtype of the output, x, residual ("" for none) and
    # weight; router and loss: dtype of the logits, `masked` the share of padding tokens
    c = dict(name=name, op=op, sources=2, tokens=128, hidden=2048, experts=128, topk=8, dtype="bf16", x="bf16",
             residual="bf16", weight="bf16", scoring="softmax", bias=False, renormalize=True, scale=1.0, masked=0.0)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one request between two layers: latency
        _case("norm_bf16_one_token", "norm", sources=1, tokens=1),
        # decoding step of two sources that dispatch in FP8: the collected sum joins the
        # residual stream and leaves as codes and scales
        _case("norm_fp8_decode", "norm", dtype="fp8"),
        # prompt processing of the same two
        _case("norm_fp8_prefill", "norm", tokens=2048, dtype="fp8"),
        # long prompts of an odd number of tokens at the wider hidden size, with the stream kept in float32
        _case("norm_bf16_float32_stream", "norm", sources=1, tokens=16381, hidden=4096, residual="fp32", weight="fp32"),
        # a training step's norm of three sources, forward and backward
        _case("norm_grad_bf16", "norm_grad", sources=3, tokens=2048),
        # the same for a float32 model of a width that no power of two divides
        _case("norm_grad_ragged", "norm_grad", sources=1, tokens=333, hidden=1160, x="fp32", residual="", weight="fp32"),
        # decoding step: every token's experts and their weights
        _case("route_softmax_decode", "route", dtype="fp32"),
        # prompts of three sources, sigmoid scores chosen with a bias per expert, padded batch
        _case("route_sigmoid_bias_prefill", "route", sources=3, tokens=2048, experts=96, topk=6, dtype="fp32",
              scoring="sigmoid", bias=True, scale=2.5, masked=0.05),
        # a training step's routes of as many sources and experts as there can be, forward and backward
        _case("route_grad_512_experts", "route_grad", sources=16, tokens=2048, experts=512, dtype="fp32",
              renormalize=False),
        # an odd batch with BF16 logits, forward and backward of the loss
        _case("balance_grad_ragged", "balance_grad", sources=1, tokens=333, experts=96, topk=6, scoring="sigmoid",
              masked=0.3),
        # training steps of two sources, and of as many as there can be
        _case("balance_grad_prefill", "balance_grad", tokens=2048, dtype="fp32", masked=0.05),
        _case("balance_grad_512_experts", "balance_grad", sources=16, tokens=2048, experts=512, dtype="fp32"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "route", "route", "route_grad", "balance_grad"])
        c = _case("", op, sources=rng.randint(1, 16), tokens=_logint(rng, 1, 4096))
        if op.startswith("norm"):
            fp8 = op == "norm" and rng.random() < 0.5
            c.update(hidden=128 * _logint(rng, 4, 64) if fp8 else 8 * _logint(rng, 32, 1024), dtype="fp8" if fp8 else "bf16",
                     x=rng.choice(["bf16", "bf16", "fp32"]), residual=rng.choice(["", "bf16", "fp32"]),
                     weight=rng.choice(["bf16", "fp32"]))
        else:
            experts = _logint(rng, 8, 512)
            c.update(experts=experts, topk=rng.randint(1, min(10, experts)), dtype=rng.choice(["bf16", "fp32"]),
                     scoring=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.7,
                     scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.05, 0.3]),
                     bias=rng.random() < 0.4 and not op.startswith("balance"))
        del c["name"]
        w = work(c)
        if w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]:
            return c


_BYTES = {"bf16": 2, "fp32": 4, "fp8": 1}


def work(case):
    n = case["sources"] * case["tokens"]
    if case["op"].startswith("norm"):
        h = case["hidden"]
        xb, yb, wb = _BYTES[case["x"]], _BYTES[case["dtype"]], _BYTES[case["weight"]]
        rb = _BYTES[case["residual"]] if case["residual"] else 0
        by = n * h * (xb + 2 * rb + yb) + h * wb      # x and the stream read, the stream and the rows written
        by += n * h // BLOCK * 4 if case["dtype"] == "fp8" else 0
        fl = n * h * 6
        if case["op"] == "norm_grad":     # another call, later: both gradients and the stream read, one written
            sb = rb or xb
            by += n * h * (yb + sb + sb + (rb and sb)) + h * (wb + 4) + 8 * n
            fl += n * h * 11
        return {"bytes": int(by), "flops": int(fl)}
    e, k, b = case["experts"], case["topk"], _BYTES[case["dtype"]]
    if case["op"] == "balance_grad":      # two calls, each of which needs every logit and id
        return {"bytes": n * e * 3 * b + 2 * n * k * 4 + e * 12, "flops": n * e * 11}
    by, fl = n * e * b + n * k * 8 + (n if case["masked"] else 0) + (4 * e if case["bias"] else 0), n * e * 5
    if case["op"] == "route_grad":
        dense = case["scoring"] == "softmax" and not case["renormalize"]      # else only the chosen ones' logits count
        by, fl = by + n * (2 * e if dense else e + k) * b + n * k * 8, fl + n * (e if dense else k) * 6
    return {"bytes": int(by), "flops": int(fl)}


# ----------------------------------------------------------------- inputs --

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, st = case["sources"] * case["tokens"], {"case": case}
    if case["op"].startswith("norm"):
        h = case["hidden"]
        st["x"] = _normal(g, (n, h)).to(_TYPES[case["x"]])
        st["weight"] = (1 + _normal(g, (h,), 0.2)).to(_TYPES[case["weight"]])
        st["residual"] = None
        if case["residual"]:      # a stream grows over the layers, in a few channels most of all
            channel = 2 * torch.exp(_normal(g, (h,), 0.7))
            st["residual"] = _normal(g, (n, h)).mul_(channel).to(_TYPES[case["residual"]])
        if case["op"] == "norm_grad":
            st["dy"] = _normal(g, (n, h), 1e-3).to(_TYPES[case["dtype"]])
            st["dstream"] = None if st["residual"] is None else _normal(g, (n, h), 1e-3).to(st["residual"].dtype)
        return st
    e, k = case["experts"], case["topk"]
    popular = _normal(g, (e,), 0.7)       # some experts are liked by every token
    st["logits"] = (_normal(g, (n, e), 1.3) + popular).to(_TYPES[case["dtype"]])
    st["bias"] = _normal(g, (e,), 0.05) - 0.05 * popular if case["bias"] else None
    st["live"] = None
    if case["masked"]:
        st["live"] = torch.rand(n, generator=g, device="cuda") >= case["masked"]
    if case["op"] == "route_grad":
        st["dweights"] = _normal(g, (n, k), 1e-2)
    if case["op"] == "balance_grad":      # the routes that the step has taken
        st["ids"] = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)[1][:, :k].int()
        if st["live"] is not None:
            st["ids"][~st["live"]] = -1
        st["dloss"] = torch.tensor(0.5, device="cuda") + 0.1 * _normal(g, ())
    return st


# -------------------------------------------------------------------- run --

def _plain_norm(st, eps):
    c, h = st["case"], st["x"].float()
    stream = None
    if st["residual"] is not None:        # what is normalised is the stream as it is kept
        stream = (h + st["residual"].float()).to(st["residual"].dtype)
        h = stream.float()
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    y = h * rstd[:, None] * st["weight"].float()
    if c["dtype"] != "fp8":
        return y.to(_TYPES[c["dtype"]]), None, stream, rstd
    s = y.reshape(len(y), -1, BLOCK).abs().amax(-1) / LARGEST
    inv = torch.where(s > 0, 1 / s, 0.0)
    return (y * inv.repeat_interleave(BLOCK, 1)).to(torch.float8_e4m3fn), s, stream, rstd


def _plain_norm_grad(st, stream, rstd):
    h = (st["x"] if stream is None else stream).float()
    dy, xhat = st["dy"].float(), h * rstd[:, None]
    a = dy * st["weight"].float()
    dh = rstd[:, None] * (a - xhat * (a * xhat).mean(1, keepdim=True))
    if st["dstream"] is not None:
        dh = dh + st["dstream"].float()
    return dh.to(st["x"].dtype if stream is None else stream.dtype), (dy * xhat).sum(0)


def _plain_scores(logits, scoring):
    """The scores in 64 bits: the choice compares them."""
    v = logits.double()
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    v = torch.exp(v - v.amax(1, keepdim=True))
    return v / v.sum(1, keepdim=True)


def _plain_route(st):
    c = st["case"]
    score = _plain_scores(st["logits"], c["scoring"])
    key = st["logits"].double() if st["bias"] is None else score + st["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["topk"]]
    w = score.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w, ids = (w * c["scale"]).float(), ids.int()
    if st["live"] is not None:
        w, ids = w * st["live"][:, None], torch.where(st["live"][:, None], ids, -1)
    return ids, w


def _plain_route_grad(st, ids):
    c, v = st["case"], st["logits"].float()
    on, at = ids >= 0, ids.clamp(min=0).long()
    dw = torch.where(on, st["dweights"], 0.0) * c["scale"]
    if c["scoring"] == "softmax":
        p = torch.exp(v - v.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-v))
    w = p.gather(1, at)
    slope = 1.0 if c["scoring"] == "softmax" else 1 - w
    if c["renormalize"]:
        q = w / w.sum(1, keepdim=True)
        d = torch.zeros_like(v).scatter_(1, at, torch.where(on, q * (dw - (dw * q).sum(1, keepdim=True)) * slope, 0.0))
    elif c["scoring"] == "sigmoid":
        d = torch.zeros_like(v).scatter_(1, at, torch.where(on, dw * w * slope, 0.0))
    else:
        d = -p * (dw * w).sum(1, keepdim=True)
        d = d.scatter_add(1, at, dw * w)
    return d.to(st["logits"].dtype)


def _plain_balance(st):
    c, v = st["case"], st["logits"].float()
    e = v.shape[1]
    on = (st["ids"] >= 0).any(1)
    counts = (st["ids"].reshape(-1, 1) == torch.arange(e, device=v.device)).sum(0).int()
    s = torch.exp(v - v.amax(1, keepdim=True)) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-v))
    p = s / s.sum(1, keepdim=True)
    n, chosen = on.sum().float(), counts.sum().float()
    slope = e * counts.float() / (chosen * n).clamp(min=1)
    loss = ((p * on[:, None]).sum(0) * slope).sum()
    d = p * (slope - (p * slope).sum(1, keepdim=True))
    if c["scoring"] == "sigmoid":
        d = d * (1 - s)
    d = torch.where(on[:, None], d * st["dloss"], 0.0)
    return loss, counts, slope, d.to(st["logits"].dtype)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import combine_layout_amd as afd
        if op.startswith("norm"):
            y = afd.rms_norm(state["x"], state["weight"], state["residual"], eps=EPS, dtype=_TYPES[c["dtype"]],
                             keep_rstd=op == "norm_grad")
            if op == "norm":
                return y.rows, y.scales, y.residual
            h = state["x"] if y.residual is None else y.residual
            dh, dweight = afd.rms_norm_grad(state["dy"], h, state["weight"], y.rstd, grad_residual=state["dstream"])
            return y.rows, y.residual, dh, dweight
        if op == "balance_grad":
            b = afd.balance_loss(state["logits"], state["ids"], scoring=c["scoring"])
            return b.loss, b.counts, afd.balance_loss_grad(state["dloss"], state["logits"], state["ids"], b.slope,
                                                           scoring=c["scoring"])
        r = afd.route_tokens(state["logits"], c["topk"], scoring=c["scoring"], bias=state["bias"],
                             renormalize=c["renormalize"], scale=c["scale"], live=state["live"])
        if op == "route":
            return r.ids, r.weights
        return r.ids, r.weights, afd.route_tokens_grad(state["dweights"], state["logits"], r.ids, scoring=c["scoring"],
                                                       renormalize=c["renormalize"], scale=c["scale"])
    if op.startswith("norm"):
        y, scales, stream, rstd = _plain_norm(state, EPS)
        return (y, scales, stream) if op == "norm" else (y, stream, *_plain_norm_grad(state, stream, rstd))
    if op == "balance_grad":
        loss, counts, _, d = _plain_balance(state)
        return loss, counts, d
    ids, w = _plain_route(state)
    return (ids, w) if op == "route" else (ids, w, _plain_route_grad(state, ids))


# ------------------------------------------------------------------ exact --

def _exact_norm(case, st):
    x, r, w = st["x"].double(), st["residual"], st["weight"].double()
    h, rounded = x, None
    if r is not None:
        rounded = (x + r.double()).to(r.dtype)     # stored in the stream's type, and normalised as stored
        h = rounded.double()
    size = torch.linalg.vector_norm(h, dim=1)
    rms = torch.sqrt(size * size / h.shape[1] + EPS)
    unit = h / rms[:, None]
    y = unit * w
    if case["op"] == "norm":
        if case["dtype"] != "fp8":
            return y, None, None if r is None else rounded.double()
        blocks = y.unflatten(1, (-1, BLOCK))
        step = blocks.abs().max(2).values / LARGEST
        codes = (blocks / torch.where(step == 0, 1.0, step)[:, :, None]).float().to(torch.float8_e4m3fn)
        return codes.flatten(1).double(), step, None if r is None else rounded.double()
    dy = st["dy"].double()
    # the derivative of h / rms(h): what is along h goes, the rest is divided by rms
    d = dy * w
    along = torch.linalg.vecdot(d, h) / (h.shape[1] * rms ** 3)
    dh = d / rms[:, None] - h * along[:, None]
    if st["dstream"] is not None:
        dh += st["dstream"].double()
    return y, None if r is None else rounded.double(), dh, torch.linalg.vecdot(dy, unit, dim=0)


def _exact_scores(case, logits):
    v = logits.double()
    return torch.softmax(v, 1) if case["scoring"] == "softmax" else torch.sigmoid(v)


def _exact_choice(case, st):
    """ids, from ranks that count the experts that come before."""
    n, e, k = st["logits"].shape[0], case["experts"], case["topk"]
    key = st["logits"].double() if st["bias"] is None else _exact_scores(case, st["logits"]) + st["bias"].double()
    ids = torch.full((n, k), -1, dtype=torch.int64, device=key.device)
    earlier = torch.arange(e, device=key.device)
    for at in range(0, n, 1024):
        block = key[at:at + 1024]
        a, b = block[:, :, None], block[:, None, :]
        rank = ((b > a) | ((b == a) & (earlier[None, :] < earlier[:, None]))).sum(2)
        row, expert = torch.nonzero(rank < k, as_tuple=True)
        ids[at + row, rank[row, expert]] = expert
    if st["live"] is not None:
        ids[~st["live"]] = -1
    return ids


def _exact_route(case, st):
    ids = _exact_choice(case, st)
    score = _exact_scores(case, st["logits"])
    on = ids >= 0
    at = torch.where(on, ids, 0)
    w = torch.where(on, torch.take_along_dim(score, at, 1), 0.0)
    total = w.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(w[:, :1])
    total = torch.where(total == 0, 1.0, total)
    weights = case["scale"] * w / total
    if case["op"] == "route":
        return ids.int(), weights
    # by the chain rule: weights from scores, then scores from logits
    dw = case["scale"] * torch.where(on, st["dweights"].double(), 0.0)
    ds = dw / total
    if case["renormalize"]:
        ds = ds - (dw * w).sum(1, keepdim=True) / total ** 2
    ds = torch.zeros_like(score).scatter_add(1, at, torch.where(on, ds, 0.0))
    if case["scoring"] == "sigmoid":
        return ids.int(), weights, ds * score * (1 - score)
    return ids.int(), weights, score * ds - score * (score * ds).sum(1, keepdim=True)


def _exact_balance(case, st):
    ids, e = st["ids"].long(), case["experts"]
    on = ids.amax(1) >= 0
    counts = torch.bincount(ids[ids >= 0], minlength=e)
    n, chosen = int(on.sum()), int(counts.sum())
    score = _exact_scores(case, st["logits"])
    total = score.sum(1, keepdim=True)
    share = score / total * on[:, None]
    slope = counts.double() * e / max(1, n * chosen)
    ds = (slope - torch.mv(share, slope)[:, None]) / total * on[:, None] * st["dloss"].double()
    if case["scoring"] == "sigmoid":
        d = ds * score * (1 - score)
    else:
        d = score * ds - score * (score * ds).sum(1, keepdim=True)
    return torch.dot(share.sum(0), slope), counts.int(), d


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    return _exact_balance(case, st) if case["op"] == "balance_grad" else _exact_route(case, st)
