"""The expert side of a round as measurable cases: products grouped by expert,
the experts' feed-forward network made of two of them, the same with low-rank
adapters of many requests, and the row tags that carry every token's adapter
to its receive rows.

``run`` computes a case in plain torch operations, or with ``own`` set through
the library's entry points.  Rows are laid out as ``worker_receive`` leaves
them: expert j of a partition owns rows [align_up(ends[j-1], alpha), ends[j]),
and the arena holds the conservative number of rows.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

SRC, RATE = 128, 448.0     # scale block, largest E4M3 value


# ------------------------------------------------------------------ cases --

def _case(name, op, **kw):
    # tokens: per source; experts: of the whole layer, split over `parts`
    # partitions, of which one is computed; inner: columns of the hidden layer
    c = dict(name=name, op=op, sources=2, tokens=128, experts=128, parts=2, topk=8, hidden=2048, inner=768, alpha=64,
             dtype="bf16", zipf=False, masked=0.0, adapters=0, rank=0, run=1)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one request through the output projection of its experts: latency
        _case("product_bf16_one_token", "product", sources=1, tokens=1, experts=96, parts=1),
        # a ragged batch of an odd number of tokens on one of three partitions, no row alignment, an odd width
        _case("product_bf16_ragged", "product", sources=1, tokens=333, experts=96, parts=3, inner=704, alpha=1,
              masked=0.05),
        # skewed routing at the wider hidden size: a few experts with most of the rows, many with few
        _case("product_fp8_skew_h4096", "product", tokens=512, hidden=4096, inner=1024, alpha=128, dtype="fp8", zipf=True),
        # decoding step of two sources: every expert's weights for some sixteen rows each
        _case("ffn_bf16_decode", "ffn"),
        # prompt processing of two sources
        _case("ffn_bf16_prefill", "ffn", tokens=2048, alpha=128),
        # three sources on one partition that holds every expert: the most arithmetic
        _case("ffn_bf16_all_experts", "ffn", sources=3, tokens=2048, experts=96, parts=1, alpha=128, masked=0.05),
        # the same two steps with FP8 activations and weights
        _case("ffn_fp8_decode", "ffn", dtype="fp8"),
        _case("ffn_fp8_prefill", "ffn", tokens=2048, alpha=128, dtype="fp8"),
        # decoding step in which every token is its own request, with one of 32 adapters
        _case("adapters_bf16_decode", "ffn", adapters=32, rank=16),
        # prompts of a few hundred tokens, each with one of 8 adapters, some with none
        _case("adapters_fp8_prefill", "ffn", tokens=2048, alpha=128, dtype="fp8", adapters=8, rank=32, run=256),
        # every token's adapter carried to its receive rows
        _case("tags_decode", "tags"),
        _case("tags_prefill", "tags", tokens=2048, alpha=128, masked=0.05),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max((work(c) for c in listed()), key=lambda w: w["flops"])
    while True:
        op = rng.choice(["product", "ffn", "ffn", "adapters", "tags"])
        experts, parts = rng.choice([(128, 2), (96, 3), (96, 1), (64, 1), (128, 4), (40, 1)])
        dtype = rng.choice(["bf16", "fp8"])
        c = _case("", "ffn" if op == "adapters" else op, sources=rng.randint(1, 3), tokens=_logint(rng, 1, 2048),
                  experts=experts, parts=parts, topk=rng.choice([1, 4, 6, 8]), hidden=256 * rng.randint(4, 16),
                  inner=128 * rng.randint(2, 10) if dtype == "fp8" else 64 * rng.randint(4, 20),
                  alpha=rng.choice([1, 16, 64, 128]), dtype=dtype, zipf=rng.random() < 0.3,
                  masked=rng.choice([0.0, 0.05, 0.3]))
        if op == "adapters":
            c.update(adapters=rng.randint(1, 32), rank=8 * rng.randint(1, 8), run=_logint(rng, 1, 512))
        del c["name"]
        w = work(c)
        if w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]:
            return c


# ----------------------------------------------------------------- routes --

def _routes(case, seed):
    """ids [N*T, K] (int64, -1 skips a choice) and every token's adapter."""
    rng = np.random.default_rng(seed)
    n, E, K = case["sources"] * case["tokens"], case["experts"], case["topk"]
    key = rng.gumbel(size=(n, E))
    if case["zipf"]:      # log-popularity plus Gumbel noise: sampling without replacement
        key = key - np.log1p(rng.permutation(E))[None, :]
    ids = np.argsort(-key, axis=1)[:, :K].astype(np.int64)
    ids[rng.random(ids.shape) < case["masked"]] = -1
    tags = np.full(n, -1, np.int64)
    if case["adapters"] or case["op"] == "tags":
        S = case["adapters"] or 32
        runs = rng.integers(-1 if case["run"] > 1 else 0, S, size=n // case["run"] + 1)   # -1: no adapter
        tags = runs[np.arange(n) // case["run"]]
    return ids, tags


def _layout(case, ids):
    """Rows of partition 0: ends [E/F], the token of every live row and its
    row number, in expert, source, token order."""
    El, a = case["experts"] // case["parts"], case["alpha"]
    ends, rows, toks, at = [], [], [], 0
    order = np.argsort(np.where((ids < 0) | (ids >= El), El, ids).reshape(-1), kind="stable")
    counts = np.bincount(ids[(ids >= 0) & (ids < El)], minlength=El)
    done = 0
    for j in range(El):
        at = -(-at // a) * a
        c = int(counts[j])
        rows.append(np.arange(at, at + c))
        toks.append(order[done:done + c] // ids.shape[1])
        done += c
        at += c
        ends.append(at)
    return np.array(ends, np.int32), np.concatenate(rows), np.concatenate(toks), counts


def _rows_cap(case):
    El = case["experts"] // case["parts"]
    return case["sources"] * case["tokens"] * min(case["topk"], El) + El * (case["alpha"] - 1)


def _shapes(case):
    """(weight rows, reduction, gated) of the case's products."""
    H, I = case["hidden"], case["inner"]
    return [(H, I, False)] if case["op"] == "product" else [(2 * I, H, True), (H, I, False)]


def work(case):
    ids, tags = _routes(case, 0)
    _, _, toks, counts = _layout(case, ids)
    R, n = len(toks), case["sources"] * case["tokens"]
    if case["op"] == "tags":
        return {"bytes": 4 * n + 4 * n * case["topk"] + 4 * R, "flops": 0}
    b = 1 if case["dtype"] == "fp8" else 2
    sc = 4 / SRC if b == 1 else 0.0
    used = int((counts > 0).sum())
    shapes = _shapes(case)
    by = used * sum(N * K * (b + sc / SRC) for N, K, _ in shapes)
    by += R * (shapes[0][1] * (b + sc) + 2 * case["hidden"])
    fl = R * sum(2 * N * K for N, K, _ in shapes)
    if case["adapters"]:
        ex = np.repeat(np.arange(len(counts)), counts)
        tg = tags[toks]
        live = tg >= 0
        pairs = len(set(zip(tg[live].tolist(), ex[live].tolist())))
        each = sum(case["rank"] * ((2 if g else 1) * K + N) for N, K, g in shapes)
        by += 2 * pairs * each + 4 * R
        fl += 2 * int(live.sum()) * each
    return {"bytes": int(by), "flops": int(fl)}


# ----------------------------------------------------------------- inputs --

def _codes(v, block_rows):
    """E4M3 codes and FP32 scales of v [..., n, k] per block_rows x 128."""
    n, k = v.shape[-2:]
    s = v.abs().reshape(*v.shape[:-2], -(-n // block_rows), min(block_rows, n), k // SRC, SRC).amax((-3, -1)) / RATE
    q = v / s.repeat_interleave(block_rows, -2)[..., :n, :].repeat_interleave(SRC, -1)
    return q.to(torch.float8_e4m3fn), s


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _inputs(case, seed):
    ids, tags = _routes(case, seed)
    ends, rows, toks, counts = _layout(case, ids)
    g = torch.Generator(device="cuda").manual_seed(seed)
    El, cap, fp8 = len(ends), _rows_cap(case), case["dtype"] == "fp8"
    st = {"ends": torch.from_numpy(ends).cuda(), "first": [int(e - c) for e, c in zip(ends, counts)],
          "last": [int(e) for e in ends]}
    x = _normal(g, (cap, _shapes(case)[0][1]), 1.0)
    st["x"], st["xs"] = _codes(x, 1) if fp8 else (x.bfloat16(), None)
    st["w"], st["ws"] = [], []
    for N, K, _ in _shapes(case):
        if fp8:
            parts = [_codes(_normal(g, (N, K), K ** -0.5), SRC) for _ in range(El)]
            st["w"].append(torch.stack([q.view(torch.uint8) for q, _ in parts]).view(torch.float8_e4m3fn))
            st["ws"].append(torch.stack([s for _, s in parts]))
        else:
            st["w"].append(torch.empty((El, N, K), dtype=torch.bfloat16, device="cuda"))
            for j in range(El):
                st["w"][-1][j] = _normal(g, (N, K), K ** -0.5)
            st["ws"].append(None)
    st["low"] = []
    if case["adapters"]:
        S, r = case["adapters"], case["rank"]
        row_tags = np.full(cap, -1, np.int32)
        row_tags[rows] = tags[toks]
        st["tags"] = torch.from_numpy(row_tags).cuda()
        for N, K, gated in _shapes(case):
            a = torch.empty((S, El, (2 if gated else 1) * r, K), dtype=torch.bfloat16, device="cuda")
            b = torch.empty((S, El, N, r), dtype=torch.bfloat16, device="cuda")
            for i in range(S):
                a[i] = _normal(g, tuple(a.shape[1:]), K ** -0.5)
                b[i] = _normal(g, tuple(b.shape[1:]), r ** -0.5)
            st["low"].append((a, b, torch.rand(S, generator=g, device="cuda") + 0.25))
    st["out"] = torch.zeros((cap, case["hidden"]), dtype=torch.bfloat16, device="cuda")
    return st


def _tag_inputs(case, seed):
    ids, tags = _routes(case, seed)
    N, T = case["sources"], case["tokens"]
    d = torch.from_numpy(ids.astype(np.int32)).cuda()
    t = torch.from_numpy(tags.astype(np.int32)).cuda()
    return {"ids": [d[s * T:(s + 1) * T] for s in range(N)], "tags": [t[s * T:(s + 1) * T] for s in range(N)],
            "out": torch.full((_rows_cap(case),), -1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    if case["op"] == "tags":
        st = _tag_inputs(case, seed)
        if own:       # a round between its receive and its reply
            import combine_layout_amd as afd
            N, T, H = case["sources"], case["tokens"], case["hidden"]
            g = torch.Generator(device="cuda").manual_seed(seed)
            buf = afd.Buffer(N, case["parts"], case["experts"], case["topk"], H, case["alpha"], T)
            for s in range(N):
                buf.source_dispatch(s, _normal(g, (T, H), 1.0).bfloat16(), st["ids"][s],
                                    torch.rand((T, case["topk"]), generator=g, device="cuda"), bucket=T)
            st["buf"], st["received"] = buf, buf.worker_receive(0, bucket=T)
    else:
        st = _inputs(case, seed)
        if own:
            import combine_layout_amd as afd
            low = [afd.LowRank(*t) for t in st["low"]]
            if case["op"] == "ffn":
                st["experts"] = afd.Experts(st["w"][0], st["w"][1], st["ws"][0], st["ws"][1])
                st["adapters"] = afd.ExpertAdapters(*low) if low else None
            st["row_tags"] = st["tags"] if low else None
    st["case"] = case
    return st


# -------------------------------------------------------------------- run --

def _wide(q, s, block_rows=1):
    """float32 values of BF16 data, or of E4M3 codes under their scales."""
    v = q.float()
    if s is None:
        return v
    return v * s.repeat_interleave(block_rows, -2)[..., :v.shape[-2], :].repeat_interleave(SRC, -1)


def _plain_product(x, w, ws, low, tags, j, gated):
    y = x @ _wide(w[j], None if ws is None else ws[j], SRC).t()
    if low is not None:
        a, b, scaling = low
        r, half = b.shape[-1], y.shape[1] // 2
        for i in range(a.shape[0]):
            on = (tags == i).float()[:, None] * scaling[i]
            t = (x @ a[i, j].float().t()) * on
            if gated:
                y[:, :half] += t[:, :r] @ b[i, j, :half].float().t()
                y[:, half:] += t[:, r:] @ b[i, j, half:].float().t()
            else:
                y += t @ b[i, j].float().t()
    if gated:
        g, u = y.chunk(2, 1)
        y = g / (1 + torch.exp(-g)) * u
    return y


def _plain_tags(case, ids, tags, out):
    El, K, a = case["experts"] // case["parts"], case["topk"], case["alpha"]
    e, t = torch.cat(ids).reshape(-1), torch.cat(tags)
    hot = (e[:, None] == torch.arange(El, device=e.device)[None, :]).int()
    rank, counts = hot.cumsum(0), hot.sum(0)
    start = ((counts + a - 1) // a * a).cumsum(0) - (counts + a - 1) // a * a
    at = torch.nonzero((e >= 0) & (e < El)).reshape(-1)
    to = start[e[at].long()] + rank[at, e[at].long()] - 1
    out[to] = t[at // K]
    return out


def run(state):
    case, out = state["case"], state["out"]
    if own:
        import combine_layout_amd as afd
        if case["op"] == "tags":
            return state["buf"].worker_tags(0, state["tags"], state["received"], out=out)
        if case["op"] == "product":
            return afd.expert_product(state["x"], state["ends"], state["w"][0], alignment=case["alpha"],
                                      x_scales=state["xs"], weight_scales=state["ws"][0], out=out)
        return afd.expert_ffn(state["x"], state["ends"], state["experts"], alignment=case["alpha"],
                              x_scales=state["xs"], adapters=state["adapters"], row_adapters=state["row_tags"], out=out)
    if case["op"] == "tags":
        return _plain_tags(case, state["ids"], state["tags"], out)
    low = state["low"] or [None, None]
    for j, (s, e) in enumerate(zip(state["first"], state["last"])):
        if s == e:
            continue
        tags = state["tags"][s:e] if state["low"] else None
        v = _wide(state["x"][s:e], None if state["xs"] is None else state["xs"][s:e])
        if case["op"] == "ffn":
            v = _plain_product(v, state["w"][0], state["ws"][0], low[0], tags, j, True)
            if case["dtype"] == "fp8":     # the hidden rows take the activations' format
                m = v.reshape(e - s, -1, SRC).abs().amax(-1) / RATE
                v = _wide((v / torch.where(m > 0, m, 1.0).repeat_interleave(SRC, 1)).to(torch.float8_e4m3fn), m)
            else:
                v = v.bfloat16().float()
        out[s:e] = _plain_product(v, state["w"][-1], state["ws"][-1], low[-1], tags, j, False).bfloat16()
    return out


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    if case["op"] == "tags":
        ids, tags = _routes(case, seed)
        _, rows, toks, _ = _layout(case, ids)
        out = torch.full((_rows_cap(case),), -1, dtype=torch.int32)
        out[torch.from_numpy(rows)] = torch.from_numpy(tags[toks].astype(np.int32))
        return out.cuda()
    st = _inputs(case, seed)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")

    def block(q, s, rows):     # [n, k] values, one 128-column slab at a time
        v = q.double()
        if s is not None:
            for i in range(s.shape[0]):
                for c in range(s.shape[1]):
                    v[i * rows:(i + 1) * rows, c * SRC:(c + 1) * SRC] *= s[i, c].double()
        return v

    def rows_of(q, s):
        v = q.double()
        return v if s is None else (v.reshape(len(v), -1, SRC) * s.double()[:, :, None]).reshape(v.shape)

    for j in range(len(st["last"])):
        sl = slice(st["first"][j], st["last"][j])
        if sl.start == sl.stop:
            continue
        v = rows_of(st["x"][sl], None if st["xs"] is None else st["xs"][sl])
        for i, (N, K, gated) in enumerate(_shapes(case)):
            w = block(st["w"][i][j], None if st["ws"][i] is None else st["ws"][i][j], SRC)
            y = torch.matmul(v, w.T.contiguous())
            if st["low"]:
                a, b, scaling = st["low"][i]
                r = case["rank"]
                for k in torch.unique(st["tags"][sl]).tolist():
                    if k < 0:
                        continue
                    at = torch.nonzero(st["tags"][sl] == k).reshape(-1)
                    for c in range(2 if gated else 1):     # gate and up each have their own pair
                        cols = slice(c * N // 2, (c + 1) * N // 2) if gated else slice(0, N)
                        full = b[k, j, cols].double() @ a[k, j, c * r:(c + 1) * r].double()
                        y[at, cols] += scaling[k].double() * torch.matmul(v[at], full.T.contiguous())
            if gated:
                y = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
                if case["dtype"] == "fp8":
                    blk = y.reshape(len(y), -1, SRC)
                    s = (blk.abs().amax(-1).float() / RATE).double()
                    q = (blk / torch.where(s > 0, s, 1.0)[:, :, None]).float().to(torch.float8_e4m3fn)
                    y = (q.double() * s[:, :, None]).reshape(y.shape)
                else:
                    y = y.bfloat16().double()
            v = y
        out[sl] = v
    return out
