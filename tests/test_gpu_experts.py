"""Grouped products, the experts' network, adapters and row tags on the GPU
against the 64-bit reference, at the counts, types and masks where they can go
wrong.  Every output buffer starts with a pattern that rows of no expert must
still hold afterwards; padding rows of x hold NaN."""
import numpy as np
import pytest
import torch

from tests import experts_ref as ref

pytestmark = pytest.mark.gpu

FILL = -7.25
ARENA = 0        # rows of the arrays where more than the case's: the host's bound picks the kernels


def _afd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_layout_amd as afd
    return afd


def _dev(t):
    if t is None:
        return None
    if t.dtype is torch.float8_e4m3fn:
        return t.view(torch.uint8).cuda().view(torch.float8_e4m3fn)
    return t.cuda()


def _low(afd, low):
    return None if low is None else afd.LowRank(*(t.cuda() for t in low))


def _check(got, want, tol, live, what):
    got = got.double().cpu()
    assert torch.equal(got[~live], torch.full_like(got[~live], FILL)), f"{what}: a row of no expert was written"
    err = (got[live] - want[live]).abs()
    bad = ~(err <= tol[live])
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, "
                           f"worst {float((err / tol[live]).nan_to_num(float('inf')).max())} of the bound")


def _widen(t, rows):
    """t on the GPU, with the arena's further rows behind it: NaN, or tag 0."""
    if t is None or ARENA <= rows:
        return _dev(t)
    if t.dtype is torch.float8_e4m3fn:
        w = torch.full((ARENA, t.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")
        w[:rows] = t.view(torch.uint8).cuda()
        return w.view(torch.float8_e4m3fn)
    w = torch.full((ARENA, *t.shape[1:]), 0 if t.dtype is torch.int32 else float("nan"), dtype=t.dtype, device="cuda")
    w[:rows] = t.cuda()
    return w


def _cut(t, rows, fill):
    """The case's rows; those behind them still hold `fill`."""
    rest = t[rows:].float()
    assert torch.equal(rest, torch.full_like(rest, fill)), "a row behind the last expert was written"
    return t[:rows]


def _run_product(afd, c, out8=False):
    n = c["w"].shape[1] // (2 if c["gated"] else 1)
    ends = torch.tensor(c["ends"], dtype=torch.int32).cuda()
    R = c["rows"]
    kw = dict(alignment=c["alpha"], x_scales=_widen(c["xs"], R), weight_scales=_dev(c["ws"]),
              activation="swiglu" if c["gated"] else None, adapters=_low(afd, c["low"]), row_adapters=_widen(c["tags"], R))
    if out8:
        out = torch.full((max(R, ARENA), n), FILL, device="cuda").to(torch.float8_e4m3fn)
        outs = torch.full((max(R, ARENA), n // 128), 1.0, device="cuda")
        afd.expert_product(_widen(c["x"], R), ends, _dev(c["w"]), out=out, out_scales=outs, **kw)
        return _cut(out, R, float(torch.tensor(FILL).to(torch.float8_e4m3fn).float())), _cut(outs, R, 1.0)
    out = torch.full((max(R, ARENA), n), FILL, dtype=torch.bfloat16, device="cuda")
    afd.expert_product(_widen(c["x"], R), ends, _dev(c["w"]), out=out, **kw)
    return _cut(out, R, FILL)


COUNTS = {
    "one_row": ([1], 1),
    "empty_and_one": ([0, 1, 0, 0, 2], 16),
    "edges": ([15, 16, 17, 0, 31, 33, 1], 1),
    "aligned": ([64, 63, 65, 0, 128, 129], 64),
    "large": ([300, 3, 513], 128),
    "many": ([(7 * i) % 11 for i in range(130)], 4),
    "tall": ([1100], 1),
    "taller": ([321, 0, 700, 256, 385], 32),       # 256-row tiles (BF16)
    "skewed": ([70, 33, 0, 17] + [0] * 60, 1),     # few rows on the average, some experts with more than a tile
}


def _print(*a):
    print("[experts]", *a, flush=True)


@pytest.mark.parametrize("shape", list(COUNTS))
@pytest.mark.parametrize("dtype,gated,k,n", [
    ("bf16", False, 256, 256), ("bf16", False, 64, 16), ("bf16", False, 704, 272), ("bf16", True, 320, 96),
    ("bf16", True, 512, 336), ("fp8", False, 128, 16), ("fp8", False, 768, 400), ("fp8", True, 384, 128),
    ("fp8", True, 256, 384)])
def test_product(shape, dtype, gated, k, n):
    afd = _afd()
    counts, alpha = COUNTS[shape]
    _print("product", shape, dtype, gated, k, n)
    c = ref.make(1, len(counts), counts, alpha, k, n * (2 if gated else 1), dtype, gated=gated)
    got = _run_product(afd, c)
    want, tol, live = ref.run_product(c, c["x"], c["xs"], c["w"], c["ws"], None, None, c["ends"], alpha, c["rows"])
    _check(got, want, ref.rounded(want, tol), live, f"{shape} {dtype}")


@pytest.mark.parametrize("shape", ["edges", "large", "taller", "skewed"])
@pytest.mark.parametrize("dtype,gated,k,n", [("bf16", False, 320, 144), ("bf16", True, 192, 80), ("fp8", False, 384, 272),
                                             ("fp8", True, 256, 256)])
def test_packed_weights_give_the_same_bits(shape, dtype, gated, k, n):
    afd = _afd()
    _print("packed", shape, dtype, gated, k, n)
    counts, alpha = COUNTS[shape]
    c = ref.make(11, len(counts), counts, alpha, k, n * (2 if gated else 1), dtype, gated=gated)
    w = _dev(c["w"])
    p = afd.pack_weights(w)
    # byte b of row r at (r / 16) * 16 * kb + (b / 16) * 256 + (r % 16) * 16 + b % 16
    E, m = w.shape[:2]
    rows = w.view(torch.uint8).reshape(E, m // 16, 16, k * w.element_size() // 16, 16)
    assert torch.equal(p.data, rows.permute(0, 1, 3, 2, 4).reshape(-1))
    kw = dict(alignment=alpha, x_scales=_widen(c["xs"], c["rows"]), weight_scales=_dev(c["ws"]),
              activation="swiglu" if gated else None)
    x, ends = _widen(c["x"], c["rows"]), torch.tensor(c["ends"], dtype=torch.int32).cuda()
    a, b = (torch.full((x.shape[0], n), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    afd.expert_product(x, ends, w, out=a, **kw)
    afd.expert_product(x, ends, p, out=b, **kw)
    assert torch.equal(a, b)


@pytest.mark.parametrize("shape", ["one_row", "edges", "aligned", "large", "many", "skewed"])
@pytest.mark.parametrize("k,n,S", [(256, 128, 0), (384, 384, 0), (256, 256, 3)])
def test_product_fp8_out(shape, k, n, S):
    afd = _afd()
    counts, alpha = COUNTS[shape]
    _print("fp8 out", shape, k, n, S)
    c = ref.make(2, len(counts), counts, alpha, k, 2 * n, "fp8", gated=True, S=S, rank=16 if S else 0)
    c["x"].view(torch.uint8)[: c["ends"][0]] = 0     # zero rows: scale 0, codes 0
    out, outs = _run_product(afd, c, out8=True)
    want, tol, live = ref.run_product(c, c["x"], c["xs"], c["w"], c["ws"], c["low"], c["tags"], c["ends"], alpha,
                                      c["rows"])
    s = outs.double().cpu()
    codes = out.float().double().cpu()
    first = slice(0, c["ends"][0])
    assert torch.equal(s[first], torch.zeros_like(s[first])) and torch.equal(codes[first], torch.zeros_like(codes[first]))
    assert torch.equal(s[~live], torch.ones_like(s[~live]))
    assert torch.equal(codes[~live], torch.full_like(codes[~live], float(torch.tensor(FILL).to(torch.float8_e4m3fn).float())))
    amax = want.abs().reshape(c["rows"], -1, 128).amax(-1)
    damax = tol.reshape(c["rows"], -1, 128).amax(-1)
    assert ((s - amax / 448).abs() <= damax / 448 + 2 * ref.F32 * (amax + damax) / 448)[live].all()
    got = codes * s.repeat_interleave(128, 1)
    step = (s * 2.0 ** -10).repeat_interleave(128, 1)
    bound = tol + (2.0 ** -4 + 4 * ref.F32) * (want.abs() + tol) + step
    assert ((got - want).abs() <= bound)[live].all()
    # every block holds its largest value as the code 448 (up to the division's rounding)
    top = codes.abs().reshape(c["rows"], -1, 128).amax(-1)
    assert (top == 448)[live & (torch.arange(c["rows"]) >= c["ends"][0])].all()


@pytest.mark.parametrize("rows", [3, 200])
def test_fp8_out_of_tiny_and_infinite_rows(rows):
    """A block whose scale would be subnormal has scale 0 and codes 0; an
    infinite value makes only its own row's block infinite."""
    afd = _afd()
    _print("tiny", rows)
    c = ref.make(12, 1, [rows], 1, 128, 256, "fp8", gated=True)
    c["xs"][0] = 2.0 ** -75          # gate and up of about 2^-75: products of about 2^-151
    c["xs"][1] = float("inf")
    out, outs = _run_product(afd, c, out8=True)
    s, codes = outs.double().cpu()[:rows], out.float().double().cpu()[:rows]
    assert s[0].item() == 0 and not codes[0].any()
    assert not torch.isfinite(s[1]).all() or torch.isnan(codes[1]).any()
    want, tol, live = ref.run_product(c, c["x"], torch.where(torch.isfinite(c["xs"]), c["xs"], torch.ones(())), c["w"],
                                      c["ws"], None, None, c["ends"], 1, c["rows"])
    got, bound = codes * s.repeat_interleave(128, 1), tol + (2.0 ** -4 + 4 * ref.F32) * (want.abs() + tol)
    bound[:rows] += (s * 2.0 ** -10).repeat_interleave(128, 1)
    assert ((got - want[:rows]).abs() <= bound[:rows])[2:].all()


@pytest.mark.parametrize("shape", ["one_row", "empty_and_one", "edges", "aligned", "large", "skewed"])
@pytest.mark.parametrize("dtype,gated,k,n,S,rank", [
    ("bf16", False, 320, 144, 1, 8), ("bf16", True, 256, 96, 5, 16), ("bf16", True, 192, 64, 40, 24),
    ("bf16", False, 256, 272, 3, 128), ("fp8", False, 256, 144, 7, 40), ("fp8", True, 384, 128, 2, 64)])
def test_adapters(shape, dtype, gated, k, n, S, rank):
    afd = _afd()
    counts, alpha = COUNTS[shape]
    _print("adapters", shape, dtype, gated, k, n, S, rank)
    c = ref.make(3, len(counts), counts, alpha, k, n * (2 if gated else 1), dtype, S=S, rank=rank, gated=gated)
    got = _run_product(afd, c)
    want, tol, live = ref.run_product(c, c["x"], c["xs"], c["w"], c["ws"], c["low"], c["tags"], c["ends"], alpha,
                                      c["rows"])
    _check(got, want, ref.rounded(want, tol), live, f"{shape} {dtype} rank {rank}")
    if S > 1:      # the adapters do something: without them the rows differ
        base = dict(c, low=None, tags=None)
        on = live & (c["tags"] >= 0) & (c["tags"] < S)
        if on.any():
            assert not torch.equal(_run_product(afd, base).cpu()[on], got.cpu()[on])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [40, 300])
def test_adapter_infinities_stay_with_their_rows(gated, rows):
    afd = _afd()
    _print("infinities", gated, rows)
    c = ref.make(4, 2, [rows, 5], 1, 256, 128 if gated else 64, "bf16", S=3, rank=16, gated=gated)
    c["low"][0][1, :, :3] = float("inf")
    c["low"][1][1, :, ::2] = float("-inf")
    c["low"][2][1] = float("nan")
    got = _run_product(afd, c)
    clean = dict(c, tags=torch.where(c["tags"] == 1, torch.tensor(-1, dtype=torch.int32), c["tags"]))
    want, tol, live = ref.run_product(clean, c["x"], None, c["w"], None, c["low"], clean["tags"], c["ends"], 1, c["rows"])
    ok = c["tags"] != 1
    err = (got.double().cpu() - want).abs()
    assert (err <= ref.rounded(want, tol))[live & ok].all()


def test_row_infinities_stay_in_their_rows():
    afd = _afd()
    _print("row infinities")
    for rows in (20, 400):
        c = ref.make(5, 2, [rows, 6], 1, 256, 64, "bf16")
        bad = torch.zeros(c["rows"], dtype=torch.bool)
        bad[::5] = True
        c["x"][bad, 3] = float("inf")
        c["x"][bad, 77] = float("nan")
        got = _run_product(afd, c).double().cpu()
        want, tol, live = ref.run_product(c, torch.where(bad[:, None], torch.zeros(()).bfloat16(), c["x"]), None, c["w"],
                                          None, None, None, c["ends"], 1, c["rows"])
        keep = live & ~bad
        assert ((got - want).abs() <= ref.rounded(want, tol))[keep].all()
        assert torch.isnan(got[live & bad]).all()


@pytest.mark.parametrize("shape", ["one_row", "edges", "aligned", "large", "tall"])
@pytest.mark.parametrize("dtype,hidden,inner,S,rank", [
    ("bf16", 256, 192, 0, 0), ("fp8", 256, 384, 0, 0), ("bf16", 512, 64, 4, 16), ("fp8", 256, 128, 6, 8)])
def test_ffn(shape, dtype, hidden, inner, S, rank):
    afd = _afd()
    counts, alpha = COUNTS[shape]
    _print("ffn", shape, dtype, hidden, inner, S, rank)
    E = len(counts)
    u = ref.make(6, E, counts, alpha, hidden, 2 * inner, dtype, S=S, rank=rank, gated=True)
    d = ref.make(7, E, counts, alpha, inner, hidden, dtype, S=S, rank=rank)
    R = u["rows"]
    out = torch.full((max(R, ARENA), hidden), FILL, dtype=torch.bfloat16, device="cuda")
    afd.expert_ffn(_widen(u["x"], R), torch.tensor(u["ends"], dtype=torch.int32).cuda(),
                   afd.Experts(_dev(u["w"]), _dev(d["w"]), _dev(u["ws"]), _dev(d["ws"])), alignment=alpha,
                   x_scales=_widen(u["xs"], R),
                   adapters=afd.ExpertAdapters(_low(afd, u["low"]), _low(afd, d["low"])) if S else None,
                   row_adapters=_widen(u["tags"], R), out=out)
    out = _cut(out, R, FILL)
    want, tol, live = ref.run_ffn(u["x"], u["xs"], u["w"], u["ws"], d["w"], d["ws"], u["low"], d["low"], u["tags"],
                                  u["ends"], alpha, u["rows"])
    _check(out, want, ref.rounded(want, tol), live, f"{shape} {dtype}")


def test_no_rows_and_ends_behind_the_rows():
    afd = _afd()
    _print("no rows")
    w = torch.randn(3, 32, 64, device="cuda").bfloat16()
    z = afd.expert_product(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"), w)
    assert z.shape == (0, 32)
    # all experts empty; ends past the rows are cut, descending ends give empty experts
    for ends in ([0, 0, 0], [50, 500, 501], [30, 10, 10], [-5, 20, 2 ** 31 - 1]):
        c = ref.make(8, 3, [20, 10, 10], 1, 64, 32, "bf16")
        c["x"] = torch.randn(c["rows"], 64).bfloat16()
        c["ends"] = ends
        got = _run_product(afd, c)
        want, tol, live = ref.run_product(c, c["x"], None, c["w"], None, None, None, ends, 1, c["rows"])
        _check(got, want, ref.rounded(want, tol), live, str(ends))


def test_rows_behind_four_gib():
    afd = _afd()
    _print("rows behind 4 GiB")
    k, n, alpha = 2048, 2304, 1 << 20
    x = torch.zeros((alpha + 5, k), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(9)
    v = torch.randn(8, k, generator=g).bfloat16()
    x[:3], x[alpha:] = v[:3].cuda(), v[3:].cuda()
    w = (torch.randn(2, n, k, generator=g) * k ** -0.5).bfloat16()
    out = torch.zeros((alpha + 5, n), dtype=torch.bfloat16, device="cuda")
    afd.expert_product(x, torch.tensor([3, alpha + 5], dtype=torch.int32).cuda(), w.cuda(), alignment=alpha, out=out)
    got = torch.cat([out[:3], out[alpha:]]).double().cpu()
    for j, sl in enumerate((slice(0, 3), slice(3, 8))):
        vd = v[sl].double()
        want, tol = ref.product(vd, torch.zeros_like(vd), w[j].double(), False, None, None, j)
        assert ((got[sl] - want).abs() <= ref.rounded(want, tol)).all()
    assert not out[3:alpha].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_graph_replays_and_two_streams(dtype):
    """A captured network with adapters replayed on new rows, routes and tags
    against eager calls, and two networks at once on two streams."""
    afd = _afd()
    _print("graph", dtype)
    hidden, inner, E, S, rank, alpha = 256, 256, 6, 3, 16, 16
    sets = []
    for seed, counts in enumerate(([20, 0, 40, 3, 16, 9], [0, 70, 1, 1, 5, 11], [30, 30, 0, 0, 0, 28])):
        u = ref.make(20 + seed, E, counts, alpha, hidden, 2 * inner, dtype, S=S, rank=rank, gated=True)
        sets.append(u)
    rows = max(s["rows"] for s in sets)
    d = ref.make(30, E, [1] * E, 1, inner, hidden, dtype, S=S, rank=rank)
    experts = afd.Experts(_dev(sets[0]["w"]), _dev(d["w"]), _dev(sets[0]["ws"]), _dev(d["ws"]))
    ad = afd.ExpertAdapters(_low(afd, sets[0]["low"]), _low(afd, d["low"]))

    def fresh():
        x = torch.zeros((rows, hidden), device="cuda").to(torch.float8_e4m3fn if dtype == "fp8" else torch.bfloat16)
        return dict(x=x, xs=torch.zeros((rows, hidden // 128), device="cuda") if dtype == "fp8" else None,
                    ends=torch.zeros(E, dtype=torch.int32, device="cuda"),
                    tags=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                    out=torch.zeros((rows, hidden), dtype=torch.bfloat16, device="cuda"))

    def load(b, s):
        n = s["rows"]
        b["x"].view(torch.uint8)[:n].copy_(_dev(s["x"]).view(torch.uint8))
        if dtype == "fp8":
            b["xs"][:n].copy_(s["xs"])
        b["ends"].copy_(torch.tensor(s["ends"], dtype=torch.int32))
        b["tags"][:n].copy_(s["tags"])
        b["out"].zero_()

    def call(b):
        afd.expert_ffn(b["x"], b["ends"], experts, alignment=alpha, x_scales=b["xs"], adapters=ad, row_adapters=b["tags"],
                       out=b["out"])

    eager, want = fresh(), []
    for s in sets:
        load(eager, s)
        call(eager)
        want.append(eager["out"].clone())
    b = fresh()
    load(b, sets[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(b)
    for i in (0, 1, 2, 0, 2):
        load(b, sets[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want[i]), f"replay of set {i}"
        load(eager, sets[(i + 1) % 3])
        call(eager)
        assert torch.equal(eager["out"], want[(i + 1) % 3])
    bufs = [fresh() for _ in range(2)]
    for b, s in zip(bufs, sets[1:]):
        load(b, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for b, st in zip(bufs, streams):
            with torch.cuda.stream(st):
                call(b)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0]["out"], want[1]) and torch.equal(bufs[1]["out"], want[2])


# ------------------------------------------------------- rounds end to end --

def _choices(ids, E):
    """(source, token, k, expert) of the valid live choices in layout order of each expert."""
    out = []
    for s, a in enumerate(ids):
        for t in range(a.shape[0]):
            for k, e in enumerate(a[t]):
                if 0 <= e < E:
                    out.append((int(e), s, t, k))
    return sorted(out)


def _ids(rng, T, E, K, masked=0.1):
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, K), np.int32)
    ids[rng.random(ids.shape) < masked] = -1
    return ids


@pytest.mark.parametrize("T,F,alpha,dispatch", [((5, 3), 2, 1, "auto"), ((0, 40), 1, 16, "auto"), ((300, 400, 1), 2, 64, "auto"),
                                                ((700, 20), 4, 8, "one_launch"), ((0, 0), 2, 1, "auto")])
@pytest.mark.parametrize("dtype,combine", [("bf16", "once"), ("fp8", "once"), ("bf16", "per_stage")])
def test_round_with_experts_and_adapters(T, F, alpha, dispatch, dtype, combine):
    """source_dispatch, worker_receive, worker_tags, worker_experts,
    worker_reply, source_collect: the tags against the sorted choices, the
    token results against the 64-bit network and the routing weights."""
    if combine != "once" and F < 2:
        pytest.skip("per stage needs two partitions")
    afd = _afd()
    _print("round", T, F, alpha, dispatch, dtype, combine)
    E, K, H, inner, S, rank = 8, 3, 256, 128, 4, 8
    rng = np.random.default_rng(5)
    N, bucket = len(T), max(max(T), 1)
    buf = afd.Buffer(N, F, E, K, H, alpha, bucket, dtype, combine=combine, dispatch=dispatch)
    x = [torch.from_numpy(rng.standard_normal((t, H), dtype=np.float32)) for t in T]
    ids = [_ids(rng, t, E, K) for t in T]
    wts = [torch.from_numpy(rng.random((t, K), dtype=np.float32)) for t in T]
    tags = [torch.from_numpy(rng.integers(-1, S, t).astype(np.int32)) for t in T]
    q = [ref.quant(v, 1) if dtype == "fp8" else (v.bfloat16(), None) for v in x]
    u = ref.make(40, E, [1] * E, 1, H, 2 * inner, dtype, S=S, rank=rank, gated=True)
    d = ref.make(41, E, [1] * E, 1, inner, H, dtype, S=S, rank=rank)
    for rnd in range(2):
        for s in range(N):
            buf.source_dispatch(s, _dev(q[s][0]), torch.from_numpy(ids[s]).cuda(), wts[s].cuda(), _dev(q[s][1]) if T[s] else None,
                                bucket=bucket)
        El = E // F
        recs = [buf.worker_receive(f, bucket=bucket) for f in range(F)]
        row_of = {}
        for f in range(F):
            got = buf.worker_tags(f, [t.cuda() for t in tags], recs[f])
            want = torch.full((recs[f].receive_rows,), -1, dtype=torch.int32)
            at, prev = 0, None
            for e, s, t, k in _choices(ids, E):
                if e // El != f:
                    continue
                if e != prev:
                    at, prev = -(-at // alpha) * alpha, e
                want[at] = tags[s][t]
                row_of[(s, t, k)] = (f, at)
                at += 1
            assert torch.equal(got.cpu(), want), f"tags of partition {f}"
            sl = slice(f * El, (f + 1) * El)
            reply = buf.worker_experts(
                f, recs[f], afd.Experts(_dev(u["w"][sl].contiguous()), _dev(d["w"][sl].contiguous()),
                                        _dev(u["ws"][sl].contiguous()) if dtype == "fp8" else None,
                                        _dev(d["ws"][sl].contiguous()) if dtype == "fp8" else None),
                adapters=afd.ExpertAdapters(
                    afd.LowRank(u["low"][0][:, sl].contiguous().cuda(), u["low"][1][:, sl].contiguous().cuda(), u["low"][2].cuda()),
                    afd.LowRank(d["low"][0][:, sl].contiguous().cuda(), d["low"][1][:, sl].contiguous().cuda(), d["low"][2].cuda())),
                row_adapters=got)
            buf.worker_reply(f, reply, recs[f].receipt)
        out = [buf.source_collect(s).double().cpu() for s in range(N)]
        for s in range(N):
            if T[s] == 0:
                continue
            want, tol, mag = (torch.zeros(T[s], H, dtype=torch.float64) for _ in range(3))
            for e in range(E):
                ts, ks = np.nonzero(ids[s] == e)
                if len(ts) == 0:
                    continue
                xv = ref.wide(q[s][0][ts], None if q[s][1] is None else q[s][1][ts])
                o, b, _ = ref.run_ffn(xv.bfloat16() if dtype == "bf16" else q[s][0][ts], None if dtype == "bf16" else q[s][1][ts],
                                      u["w"][e:e + 1], u["ws"][e:e + 1] if dtype == "fp8" else None, d["w"][e:e + 1],
                                      d["ws"][e:e + 1] if dtype == "fp8" else None,
                                      tuple(t[:, e:e + 1] if t.dim() > 1 else t for t in u["low"]),
                                      tuple(t[:, e:e + 1] if t.dim() > 1 else t for t in d["low"]), tags[s][ts],
                                      [len(ts)], 1, len(ts))
                w = wts[s][ts, ks].double()[:, None]
                want[ts] += w * o
                tol[ts] += w * ref.rounded(o, b)
                mag[ts] += w * (o.abs() + ref.rounded(o, b))
            tol = tol + 2 * K * ref.F32 * mag
            if combine == "per_stage":   # every partial is rounded to BF16; their magnitudes sum to at most mag
                tol = tol + (ref.BF16 + F * ref.F32) * mag
            assert ((out[s] - want).abs() <= ref.rounded(want, tol)).all(), f"round {rnd} source {s}"


def test_tags_keep_rows_of_no_choice_and_refusals():
    afd = _afd()
    _print("tags refusals")
    buf = afd.Buffer(1, 2, 4, 2, 256, 16, 8)
    ids = torch.tensor([[0, 3], [-1, 1], [2, -1]], dtype=torch.int32).cuda()
    buf.source_dispatch(0, torch.zeros((3, 256), dtype=torch.bfloat16).cuda(), ids, torch.ones((3, 2)).cuda(), bucket=8)
    recs = [buf.worker_receive(f, bucket=8) for f in range(2)]
    tags = torch.tensor([5, 6, 7], dtype=torch.int32).cuda()
    out = torch.full((recs[0].receive_rows,), 99, dtype=torch.int32, device="cuda")
    assert buf.worker_tags(0, [tags], recs[0], out=out) is out
    want = torch.full_like(out, 99).cpu()
    want[0], want[16] = 5, 6
    assert torch.equal(out.cpu(), want)
    for bad in ([tags[:2]], [tags.long()], [tags.cpu()], [None], [tags, tags], []):
        with pytest.raises(ValueError):
            buf.worker_tags(0, bad, recs[0])
    with pytest.raises(ValueError):
        buf.worker_tags(0, [tags], recs[0], out=out[:-1])
    with pytest.raises(afd.AfdError):
        buf.worker_tags(1, [tags], recs[0])      # a receipt of another partition
    with pytest.raises(ValueError):
        buf.worker_experts(1, recs[0], None)
    for f in range(2):
        buf.worker_reply(f, torch.zeros((recs[f].receive_rows, 256), dtype=torch.bfloat16, device="cuda"), recs[f].receipt)
    with pytest.raises(afd.AfdError):
        buf.worker_tags(0, [tags], recs[0])      # after the reply


def test_tags_of_a_cached_round():
    """A round that reuses the last layout has its slot map: tags follow it."""
    afd = _afd()
    _print("tags cached")
    rng = np.random.default_rng(3)
    T, E, K, F, alpha = 50, 8, 3, 2, 4
    ids = _ids(rng, T, E, K)
    buf = afd.Buffer(1, F, E, K, 256, alpha, T)
    first = []
    for rnd in range(2):
        x = torch.randn(T, 256, device="cuda").bfloat16()
        buf.source_dispatch(0, x, torch.from_numpy(ids).cuda() if rnd == 0 else None, torch.rand(T, K, device="cuda"), bucket=T,
                            cached=rnd > 0)
        recs = [buf.worker_receive(f, bucket=T) for f in range(F)]
        tags = torch.arange(T, dtype=torch.int32, device="cuda") * (rnd + 1)
        got = [buf.worker_tags(f, [tags], recs[f]) for f in range(F)]
        if rnd == 0:
            first = [g.clone() for g in got]
        else:
            for f in range(F):
                assert torch.equal(got[f], torch.where(first[f] >= 0, first[f] * 2, first[f]))
        for f in range(F):
            live = got[f] >= 0      # the token's row stands where its tag does
            tok = (got[f][live] // (rnd + 1)).long()
            assert torch.equal(recs[f].rows[live], x[tok])
            buf.worker_reply(f, torch.zeros((recs[f].receive_rows, 256), dtype=torch.bfloat16, device="cuda"), recs[f].receipt)
        buf.source_collect(0)


def test_python_refusals():
    afd = _afd()
    _print("refusals")
    x = torch.zeros((8, 128), dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([4, 8], dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 32, 128), dtype=torch.bfloat16, device="cuda")
    xq, xs = x.to(torch.float8_e4m3fn), torch.ones((8, 1), device="cuda")
    wq, ws = w.to(torch.float8_e4m3fn), torch.ones((2, 1, 1), device="cuda")
    low = afd.LowRank(torch.zeros((3, 2, 8, 128), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((3, 2, 32, 8), dtype=torch.bfloat16, device="cuda"), torch.ones(3, device="cuda"))
    tags = torch.zeros(8, dtype=torch.int32, device="cuda")
    afd.expert_product(x, ends, w)
    afd.expert_product(xq, ends, wq, x_scales=xs, weight_scales=ws)
    afd.expert_product(x, ends, w, adapters=low, row_adapters=tags)
    bad = [
        (TypeError, (x.float(), ends, w), {}), (ValueError, (x.cpu(), ends, w), {}), (ValueError, (x.t(), ends, w), {}),
        (ValueError, (x[0], ends, w), {}), (ValueError, (x, ends.long(), w), {}), (ValueError, (x, ends[:1], w), {}),
        (ValueError, (x, ends.cpu(), w), {}), (ValueError, (x, ends, w.float()), {}), (ValueError, (x, ends, w[:, :, :64]), {}),
        (ValueError, (x, ends, w[0]), {}), (ValueError, (x, ends, w.cpu()), {}), (ValueError, (x, ends, w), dict(activation="gelu")),
        (ValueError, (x, ends, w[:, :31].contiguous()), dict(activation="swiglu")),
        (ValueError, (x, ends, w), dict(x_scales=xs)), (ValueError, (x, ends, w), dict(weight_scales=ws)),
        (ValueError, (xq, ends, wq), {}), (ValueError, (xq, ends, wq), dict(x_scales=xs)),
        (ValueError, (xq, ends, wq), dict(x_scales=xs[:4], weight_scales=ws)),
        (ValueError, (x, ends, w), dict(row_adapters=tags)), (ValueError, (x, ends, w), dict(adapters=low)),
        (ValueError, (x, ends, w), dict(adapters=low, row_adapters=tags[:4])),
        (ValueError, (x, ends, w), dict(adapters=low._replace(a=low.a[:2]), row_adapters=tags)),
        (ValueError, (x, ends, w), dict(adapters=low._replace(scaling=low.scaling[0]), row_adapters=tags)),
        (ValueError, (x, ends, w), dict(out=torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda"))),
        (ValueError, (x, ends, w), dict(out=torch.zeros((8, 32), device="cuda"))),
        (ValueError, (x, ends, w), dict(out_scales=xs)),
        (ValueError, (x.clone().requires_grad_(), ends, w), {}), (ValueError, (x, ends, w.clone().requires_grad_()), {}),
        (ValueError, (x, ends, w), dict(alignment=0)), (ValueError, (x, ends, w), dict(alignment=2 ** 32 + 1)),
        (afd.AfdError, (x[:, :32].contiguous(), ends, w[:, :, :32].contiguous()), {}),
        (afd.AfdError, (x, ends, w[:, :24].contiguous()), {}),
        (afd.AfdError, (x, ends, w), dict(out=torch.zeros((8, 32), device="cuda").to(torch.float8_e4m3fn), out_scales=xs)),
    ]
    for err, args, kw in bad:
        with pytest.raises((err, ValueError) if err is afd.AfdError else err):
            afd.expert_product(*args, **kw)
    with torch.no_grad():
        afd.expert_product(x.clone().requires_grad_(), ends, w)
    up, down = torch.zeros((2, 128, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 128, 64), dtype=torch.bfloat16, device="cuda")
    ex = afd.Experts(up, down)
    assert afd.expert_ffn(x, ends, ex).shape == (8, 128)
    with pytest.raises(ValueError):
        afd.expert_ffn(x, ends[:1], ex)
    with pytest.raises(ValueError):
        afd.expert_ffn(x, ends, ex, alignment=2 ** 32)
    with pytest.raises(ValueError):
        afd.expert_ffn(xq, ends, ex, x_scales=xs)
    with pytest.raises(ValueError):
        afd.expert_ffn(x, ends, afd.Experts(up, up))
    with pytest.raises(ValueError):
        afd.pack_weights(up.cpu())
    with pytest.raises(ValueError):
        afd.pack_weights(up.transpose(1, 2))
    with pytest.raises(afd.AfdError):
        afd.pack_weights(torch.zeros((1, 20, 64), dtype=torch.bfloat16, device="cuda"))


def test_a_stream_that_is_not_the_default():
    """Inputs made on one stream and used, in order, on another."""
    afd = _afd()
    _print("side stream")
    c = ref.make(13, 3, [40, 0, 90], 1, 256, 64, "bf16", S=2, rank=16)
    want = _run_product(afd, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run_product(afd, c)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


# The products choose between two kernels by the host's bound of the rows.  The cases
# above leave most of these small sizes to the few-row kernel; in an arena of many rows
# (its first ones used) the tiled kernel computes them.

@pytest.fixture
def arena(monkeypatch):
    monkeypatch.setitem(globals(), "ARENA", 32 * 2100)


TILED = ["one_row", "edges", "aligned", "large", "many", "tall", "taller", "skewed"]


@pytest.mark.parametrize("shape", TILED)
@pytest.mark.parametrize("dtype,gated,k,n", [
    ("bf16", False, 64, 16), ("bf16", False, 704, 272), ("bf16", True, 320, 96), ("bf16", True, 512, 336),
    ("fp8", False, 128, 16), ("fp8", False, 768, 400), ("fp8", True, 384, 128), ("fp8", True, 256, 384)])
def test_product_in_an_arena(arena, shape, dtype, gated, k, n):
    test_product(shape, dtype, gated, k, n)


@pytest.mark.parametrize("shape", ["edges", "large", "taller"])
@pytest.mark.parametrize("dtype,gated,k,n", [("bf16", False, 320, 144), ("bf16", True, 192, 80), ("fp8", False, 384, 272),
                                             ("fp8", True, 256, 256)])
def test_packed_weights_in_an_arena(arena, shape, dtype, gated, k, n):
    test_packed_weights_give_the_same_bits(shape, dtype, gated, k, n)


@pytest.mark.parametrize("shape", ["one_row", "edges", "aligned", "large", "many", "skewed"])
@pytest.mark.parametrize("k,n,S", [(256, 128, 0), (384, 384, 0), (256, 256, 3)])
def test_product_fp8_out_in_an_arena(arena, shape, k, n, S):
    test_product_fp8_out(shape, k, n, S)


@pytest.mark.parametrize("shape", ["one_row", "empty_and_one", "edges", "aligned", "large", "skewed"])
@pytest.mark.parametrize("dtype,gated,k,n,S,rank", [
    ("bf16", False, 320, 144, 1, 8), ("bf16", True, 256, 96, 5, 16), ("bf16", True, 192, 64, 40, 24),
    ("bf16", False, 256, 272, 3, 128), ("fp8", False, 256, 144, 7, 40), ("fp8", True, 384, 128, 2, 64)])
def test_adapters_in_an_arena(arena, shape, dtype, gated, k, n, S, rank):
    test_adapters(shape, dtype, gated, k, n, S, rank)


@pytest.mark.parametrize("shape", ["one_row", "edges", "aligned", "large", "tall"])
@pytest.mark.parametrize("dtype,hidden,inner,S,rank", [
    ("bf16", 256, 192, 0, 0), ("fp8", 256, 384, 0, 0), ("bf16", 512, 64, 4, 16), ("fp8", 256, 128, 6, 8)])
def test_ffn_in_an_arena(arena, shape, dtype, hidden, inner, S, rank):
    test_ffn(shape, dtype, hidden, inner, S, rank)


def test_infinities_in_an_arena(arena):
    for gated in (False, True):
        test_adapter_infinities_stay_with_their_rows(gated, 300)
    test_row_infinities_stay_in_their_rows()
    test_fp8_out_of_tiny_and_infinite_rows(200)


def test_tiled_rows_behind_four_gib():
    """The tiled kernel across 4 GiB of x: rows of zeros but for the first and last."""
    afd = _afd()
    _print("tiled rows behind 4 GiB")
    k, n, many = 2048, 2304, (1 << 20) + 5
    x = torch.zeros((many, k), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(9)
    v = torch.randn(8, k, generator=g).bfloat16()
    x[:3], x[-5:] = v[:3].cuda(), v[3:].cuda()
    w = (torch.randn(2, n, k, generator=g) * k ** -0.5).bfloat16()
    out = torch.full((many, n), FILL, dtype=torch.bfloat16, device="cuda")
    afd.expert_product(x, torch.tensor([3, many], dtype=torch.int32).cuda(), w.cuda(), out=out)
    got = torch.cat([out[:3], out[-5:]]).double().cpu()
    for j, sl in enumerate((slice(0, 3), slice(3, 8))):
        vd = v[sl].double()
        want, tol = ref.product(vd, torch.zeros_like(vd), w[j].double(), False, None, None, j)
        assert ((got[sl] - want).abs() <= ref.rounded(want, tol)).all()
    assert not out[3:-5].any()


@pytest.mark.parametrize("S", [0, 3])
def test_network_into_its_own_rows(S):
    """The network's rows may take the place of x; a single product refuses that."""
    afd = _afd()
    _print("in place", S)
    counts, alpha = COUNTS["aligned"]
    E, H, inner = len(counts), 256, 128
    u = ref.make(14, E, counts, alpha, H, 2 * inner, "bf16", S=S, rank=8 if S else 0, gated=True)
    d = ref.make(15, E, counts, alpha, inner, H, "bf16", S=S, rank=8 if S else 0)
    x, ends = u["x"].cuda(), torch.tensor(u["ends"], dtype=torch.int32).cuda()
    kw = dict(alignment=alpha, row_adapters=_dev(u["tags"]),
              adapters=afd.ExpertAdapters(_low(afd, u["low"]), _low(afd, d["low"])) if S else None)
    ex = afd.Experts(u["w"].cuda(), d["w"].cuda())
    want = afd.expert_ffn(x, ends, ex, **kw)
    got = afd.expert_ffn(x, ends, ex, out=x, **kw)
    live = u["live"].cuda()
    assert got.data_ptr() == x.data_ptr() and torch.equal(got[live], want[live])
    assert torch.isnan(x[~live]).all()
    square = torch.zeros((E, H, H), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(afd.AfdError):
        afd.expert_product(x, ends, square, alignment=alpha, out=x)
