"""The network against its own two products: expert_ffn gives the bits of the
gated product into hidden rows and the second product of these, and the second
product's values, from hidden rows that are then known exactly, lie within a
BF16 rounding and float32 and matrix-unit sums of the 64-bit ones (a bound that
passes through the hidden rows' own rounding is far wider).  Both kernels: in
the case's rows and in an arena of many."""
import pytest
import torch

from tests import experts_bounds as bounds
from tests import experts_ref as ref
from tests.test_gpu_experts import COUNTS, FILL, _afd, _dev, _low, _print

pytestmark = pytest.mark.gpu

ARENA = 32 * 2100       # rows of an arena for which the tiled kernel is chosen


def _wide(t, rows, fill):
    """t on the GPU with rows of `fill` bytes behind it."""
    if t is None:
        return None
    w = torch.full((rows, *t.shape[1:]), fill, dtype=torch.uint8, device="cuda") if t.element_size() == 1 else \
        torch.full((rows, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
    w[:t.shape[0]] = t.view(torch.uint8).cuda() if t.element_size() == 1 else t.cuda()
    return w.view(t.dtype)


@pytest.mark.parametrize("arena", [False, True])
@pytest.mark.parametrize("shape", ["one_row", "edges", "aligned", "large", "tall"])
@pytest.mark.parametrize("dtype,hidden,inner,S,rank", [
    ("bf16", 256, 192, 0, 0), ("fp8", 256, 384, 0, 0), ("bf16", 512, 64, 4, 16), ("fp8", 256, 128, 6, 8),
    ("fp8", 128, 256, 0, 0), ("bf16", 64, 320, 3, 8)])
def test_network_is_its_two_products(arena, shape, dtype, hidden, inner, S, rank):
    afd = _afd()
    counts, alpha = COUNTS[shape]
    _print("two products", arena, shape, dtype, hidden, inner, S, rank)
    E, fp8 = len(counts), dtype == "fp8"
    u = ref.make(16, E, counts, alpha, hidden, 2 * inner, dtype, S=S, rank=rank, gated=True)
    d = ref.make(17, E, counts, alpha, inner, hidden, dtype, S=S, rank=rank)
    d["tags"] = u["tags"]
    R = ARENA if arena else u["rows"]
    x, xs, tags = _wide(u["x"], R, 0x7F if fp8 else float("nan")), _wide(u["xs"], R, 1.0), _wide(u["tags"], R, 0)
    ends = torch.tensor(u["ends"], dtype=torch.int32).cuda()
    up, down, ups, downs = _dev(u["w"]), _dev(d["w"]), _dev(u["ws"]), _dev(d["ws"])
    lu, ld = _low(afd, u["low"]), _low(afd, d["low"])
    h = torch.full((R, inner), 0.5, device="cuda").to(x.dtype)
    hs = torch.full((R, inner // 128), 1.0, device="cuda") if fp8 else None
    one, two = (torch.full((R, hidden), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kw = dict(alignment=alpha, row_adapters=tags if S else None)
    afd.expert_product(x, ends, afd.pack_weights(up), x_scales=xs, weight_scales=ups, activation="swiglu", adapters=lu,
                       out=h, out_scales=hs, **kw)
    afd.expert_product(h, ends, afd.pack_weights(down), x_scales=hs, weight_scales=downs, adapters=ld, out=two, **kw)
    afd.expert_ffn(x, ends, afd.Experts(up, down, ups, downs), x_scales=xs,
                   adapters=afd.ExpertAdapters(lu, ld) if S else None, out=one, **kw)
    assert torch.equal(one, two)
    n, live = u["rows"], u["live"]
    got = one.double().cpu()
    assert (got[n:] == FILL).all() and (got[:n][~live] == FILL).all()
    hc = h.cpu()[:n] if not fp8 else h.view(torch.uint8).cpu()[:n].view(torch.float8_e4m3fn)
    want, tol, _ = bounds.product(d, hc, hs.cpu()[:n] if fp8 else None, d["low"], d["w"], d["ws"])
    bad = ~((got[:n] - want).abs() <= ref.rounded(want, tol))[live]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off"


@pytest.mark.parametrize("arena", [False, True])
@pytest.mark.parametrize("rows,n,k", [(3, 16, 128), (40, 272, 256), (200, 144, 384)])
def test_fp8_sums_of_cancelling_products(arena, rows, n, k):
    """Codes over E4M3's whole range, most of whose products cancel: what is left
    of the sums is as small as what the matrix unit loses."""
    afd = _afd()
    _print("cancelling", arena, rows, n, k)
    g = torch.Generator().manual_seed(18)

    def codes(r):
        v = torch.exp2(torch.rand(r, k, generator=g) * 17 - 9) * torch.sign(torch.randn(r, k, generator=g))
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).float()

    x, w = codes(rows), codes(n)
    # three quarters of the columns come in pairs of equal codes in w and opposite ones in x
    at = torch.randperm(k, generator=g)[:k // 4 * 3]
    a, b = at[:len(at) // 2], at[len(at) // 2:]
    x[:, b], w[:, b] = -x[:, a], w[:, a]
    xq, wq = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    xs = torch.exp2(torch.randint(-3, 4, (rows, k // 128), generator=g).float())
    ws = torch.exp2(torch.randint(-3, 4, (1, (n + 127) // 128, k // 128), generator=g).float())
    R = ARENA if arena else rows
    got = afd.expert_product(_wide(xq, R, 0x7F), torch.tensor([rows], dtype=torch.int32).cuda(), _dev(wq[None].contiguous()),
                             x_scales=_wide(xs, R, 1.0), weight_scales=ws.cuda())[:rows].double().cpu()
    case = dict(tags=None, ends=[rows], alpha=1, rows=rows)
    want, tol, _ = bounds.product(case, xq, xs, None, wq[None], ws)
    assert ((got - want).abs() <= ref.rounded(want, tol)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,F,alpha", [((5, 3), 2, 1), ((0, 40), 1, 16), ((300, 400, 1), 4, 64)])
def test_round_is_its_replies(dtype, T, F, alpha):
    """A round's replies are expert_ffn of its received rows, bit for bit, and its
    results are the replies' weighted sums within float32 and one BF16 rounding
    (the tags name every row's source and token)."""
    afd = _afd()
    _print("round", dtype, T, F, alpha)
    E, K, H, inner, S, rank = 8, 3, 256, 128, 4, 8
    g = torch.Generator().manual_seed(24)
    N, bucket, El = len(T), max(T), E // F
    u = ref.make(25, E, [1] * E, 1, H, 2 * inner, dtype, S=S, rank=rank, gated=True)
    d = ref.make(26, E, [1] * E, 1, inner, H, dtype, S=S, rank=rank)
    buf = afd.Buffer(N, F, E, K, H, alpha, bucket, dtype)
    first = [sum(T[:s]) for s in range(N)]
    for s in range(N):
        x = torch.randn(T[s], H, generator=g)
        q, qs = (ref.quant(x, 1) if dtype == "fp8" else (x.bfloat16(), None)) if T[s] else (None, None)
        ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T[s])]).int() if T[s] else torch.zeros(0, K).int()
        ids[torch.rand(ids.shape, generator=g) < 0.1] = -1
        buf.source_dispatch(s, _dev(q), ids.cuda(), torch.rand(T[s], K, generator=g).cuda(), _dev(qs), bucket=bucket)
    token = [torch.arange(first[s], first[s] + T[s], dtype=torch.int32, device="cuda") for s in range(N)]
    adapter = [torch.randint(-1, S, (t,), generator=g).int().cuda() for t in T]
    want, mag = (torch.zeros(sum(T), H, dtype=torch.float64, device="cuda") for _ in range(2))
    recs = [buf.worker_receive(f, bucket=bucket) for f in range(F)]
    for f, rec in enumerate(recs):
        sl = slice(f * El, (f + 1) * El)
        cut = lambda t: None if t is None else _dev(t[sl].contiguous())   # noqa: E731
        ex = afd.Experts(cut(u["w"]), cut(d["w"]), cut(u["ws"]), cut(d["ws"]))
        ad = afd.ExpertAdapters(*(afd.LowRank(c["low"][0][:, sl].contiguous().cuda(), c["low"][1][:, sl].contiguous().cuda(),
                                              c["low"][2].cuda()) for c in (u, d)))
        tags, rows = buf.worker_tags(f, adapter, rec), buf.worker_tags(f, token, rec).long()
        reply = buf.worker_experts(f, rec, ex, adapters=ad, row_adapters=tags)
        again = afd.expert_ffn(rec.rows, rec.ends, ex, alignment=alpha, x_scales=rec.scales, adapters=ad, row_adapters=tags,
                               rows_per_expert=-(-sum(T) * K // E))
        live = rows >= 0
        assert torch.equal(reply[live], again[live])
        part = rec.weights[live].double()[:, None] * reply[live].double()
        want.index_add_(0, rows[live], part)
        mag.index_add_(0, rows[live], part.abs())
        buf.worker_reply(f, reply, rec.receipt)
    for s in range(N):
        got = buf.source_collect(s).double()
        at = slice(first[s], first[s] + T[s])
        # K products and K sums in float32, then BF16
        assert ((got - want[at]).abs() <= ref.rounded(want[at], 2 * K * ref.F32 * mag[at])).all(), f"source {s}"
