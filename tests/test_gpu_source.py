"""The source's side on the GPU against its 64-bit reference, at the sizes, types
and masks where it can go wrong."""
import pytest
import torch

from tests import source_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


def _afd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_layout_amd as afd
    return afd


def _print(*a):
    print("[source]", *a, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def _gapped(t, gap):
    """t on the GPU with `gap` columns of NaN behind every row."""
    if not gap:
        return t.cuda()
    w = torch.full((t.shape[0], t.shape[1] + gap), NAN, dtype=t.dtype, device="cuda")
    w[:, :t.shape[1]] = t.cuda()
    return w[:, :t.shape[1]]


# -------------------------------------------------------------------- norm --

def _norm_case(seed, T, H, xt, rt, wt):
    g = _gen(seed)
    x, w = _rand(g, T, H, dtype=xt), (1 + _rand(g, H, std=0.3)).to(wt)
    r = None if rt is None else _rand(g, T, H, std=4.0, dtype=rt)
    if T > 2:
        x[1] = 0
        if r is not None:
            r[1] = 0
    return x, r, w


WIDTHS = [8, 24, 128, 512, 520, 1024, 1160, 2048, 2056, 4096, 5000, 8192, 8200, 12000, 16376, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("xt,rt,wt,T", [(BF, BF, BF, 5), (BF, F32, F32, 3), (F32, None, F32, 6), (BF, None, BF, 1),
                                        (F32, BF, BF, 2), (F32, F32, BF, 9)])
def test_norm(H, xt, rt, wt, T):
    afd = _afd()
    _print("norm", H, xt, rt, wt, T)
    x, r, w = _norm_case(H + T, T, H, xt, rt, wt)
    n = afd.rms_norm(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=1e-5, keep_rstd=True)
    h, rstd, y, rel = ref.norm(x, w, r, 1e-5)
    assert n.scales is None
    if r is None:
        assert n.residual is None
    else:
        assert n.residual.dtype is rt and torch.equal(n.residual.double().cpu(), h)
    ref.check(n.rstd, rstd, (rel + ref.U) * rstd, "rstd")
    ref.check(n.rows, y, ref.rounded(y, (rel + 3 * ref.U) * y.abs(), BF), "rows")
    assert n.rows.dtype is BF and n.rows.is_contiguous()


@pytest.mark.parametrize("H", [128, 384, 1024, 2048, 4096, 5120, 8192, 12288, 16384])
@pytest.mark.parametrize("xt,rt,wt,T", [(BF, BF, BF, 5), (BF, None, F32, 3), (F32, F32, BF, 4), (BF, F32, F32, 1)])
def test_norm_fp8(H, xt, rt, wt, T):
    afd = _afd()
    _print("norm fp8", H, xt, rt, wt, T)
    x, r, w = _norm_case(3 * H + T, T, H, xt, rt, wt)
    w[:64] = 0                                       # half a block of zeros
    n = afd.rms_norm(x.cuda(), w.cuda(), None if r is None else r.cuda(), dtype=F8)
    h, rstd, y, rel = ref.norm(x, w, r, 1e-6)
    if r is not None:
        assert torch.equal(n.residual.double().cpu(), h)
    amax = y.abs().reshape(T, -1, 128).amax(-1)
    s = n.scales.double().cpu()
    rel = rel + 3 * ref.U
    ref.check(n.scales, amax / 448, (rel + 2 * ref.U) * amax / 448, "scales")
    if T > 2:
        assert (s[1] == 0).all() and (n.rows[1].float() == 0).all()
    wide = s.repeat_interleave(128, 1)
    got = n.rows.float().double().cpu() * wide
    # the code is off by half a step of its value, or of the smallest one's; its factor by two more roundings
    tol = rel * y.abs() + (2.0 ** -4 + 4 * ref.U) * y.abs() * (1 + rel) + wide * 2.0 ** -10
    ref.check(got, y, tol, "codes")
    top = n.rows.float().abs().cpu().reshape(T, -1, 128).amax(-1)
    assert (top[s > 0] == 448).all()


def test_norm_fp8_takes_the_dispatch_format():
    """Scales as the exchange's experts make them: a block below float32's normal range is 0."""
    afd = _afd()
    x = torch.ones(2, 256, device="cuda")
    w = torch.full((256,), 1e-37, device="cuda")
    w[128:] = 6e-36
    n = afd.rms_norm(x, w, dtype=F8, eps=1e-6)
    assert (n.scales[:, 0] == 0).all() and (n.rows[:, :128].float() == 0).all()
    assert (n.scales[:, 1] > 0).all() and (n.rows[:, 128:].float() == 448).all()


@pytest.mark.parametrize("T", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("H,gap", [(256, 8), (2048, 16), (4096, 0), (2048, 0)])
def test_norm_strides_and_rows(T, H, gap):
    afd = _afd()
    _print("norm strides", T, H, gap)
    x, r, w = _norm_case(T, T, H, BF, BF, BF)
    want = afd.rms_norm(x.cuda(), w.cuda(), r.cuda(), keep_rstd=True)
    ro = _gapped(torch.zeros_like(r), gap)
    got = afd.rms_norm(_gapped(x, gap), w.cuda(), _gapped(r, 2 * gap), residual_out=ro, keep_rstd=True)
    assert got.residual is ro
    for a, b in zip(want, got):
        assert a is None and b is None or torch.equal(a, b)
    if gap and T > 1:
        assert ro._base[:, H:].isnan().all()


def test_norm_in_place():
    afd = _afd()
    for rt, xt in ((BF, BF), (F32, BF), (F32, F32)):
        x, r, w = (t.cuda() for t in _norm_case(7, 70, 2048, xt, rt, BF))
        want = afd.rms_norm(x, w, r)
        s = r.clone()
        got = afd.rms_norm(x, w, s, residual_out=s)           # the stream where it stands
        assert got.residual is s and torch.equal(s, want.residual) and torch.equal(got.rows, want.rows)
        if xt is rt:
            s = x.clone()
            got = afd.rms_norm(s, w, r, residual_out=s)       # the stream over x
            assert torch.equal(s, want.residual) and torch.equal(got.rows, want.rows)
        if xt is BF:
            s, q = x.clone(), r.clone()
            got = afd.rms_norm(s, w, q, residual_out=q, out=s)
            assert torch.equal(s, want.rows) and torch.equal(q, want.residual)
    y = afd.rms_norm(x.bfloat16(), w)
    s = x.bfloat16()
    assert torch.equal(afd.rms_norm(s, w, out=s).rows, y.rows)


def test_norm_rows_do_not_reach_each_other():
    """Infinities and NaNs stay in their rows, and in FP8 in their blocks; rows behind the last are left."""
    afd = _afd()
    for H, dtype in ((2048, BF), (4096, BF), (2048, F8), (8192, F8)):
        x, r, w = (t.cuda() for t in _norm_case(3, 9, H, BF, BF, BF))
        clean = afd.rms_norm(x, w, r, dtype=dtype)
        x[2, 5], x[4, 7], r[6, 300] = INF, NAN, -INF
        out = torch.full((12, H), 3.0, device="cuda").to(dtype)
        scales = torch.full((12, H // 128), 3.0, device="cuda") if dtype is F8 else None
        ro = torch.full((12, H), 3.0, dtype=BF, device="cuda")
        n = afd.rms_norm(x, w, r, dtype=dtype, out=out[:9], out_scales=None if scales is None else scales[:9],
                         residual_out=ro[:9])
        keep = [0, 1, 3, 5, 7, 8]
        assert torch.equal(n.rows[keep].float(), clean.rows[keep].float())
        assert torch.equal(n.residual[keep], clean.residual[keep])
        assert n.residual[2, 5] == INF and n.residual[4, 7].isnan() and n.residual[6, 300] == -INF
        assert (out[9:].float() == 3).all() and (ro[9:] == 3).all() and (scales is None or (scales[9:] == 3).all())
        assert n.rows[4].float().isnan().any()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("ht,wt,T,res", [(BF, BF, 5, True), (F32, F32, 3, True), (F32, BF, 1, False), (BF, F32, 70, False)])
def test_norm_grad(H, ht, wt, T, res):
    afd = _afd()
    _print("norm grad", H, ht, wt, T, res)
    g = _gen(H + T)
    h, w = _rand(g, T, H, std=2.0, dtype=ht), (1 + _rand(g, H, std=0.3)).to(wt)
    dy, dr = _rand(g, T, H, dtype=BF), _rand(g, T, H, dtype=ht) if res else None
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dh, dw = afd.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(),
                               grad_residual=None if dr is None else dr.cuda())
    want, tol, wantw, tolw = ref.norm_grad(dy.double(), h.double(), w.double(), rstd.double(),
                                           None if dr is None else dr.double())
    ref.check(dh, want, ref.rounded(want, tol, ht), "dh")
    ref.check(dw, wantw, tolw + ref.U * wantw.abs(), "dweight")
    assert dh.dtype is ht and dw.dtype is F32
    again = afd.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), grad_residual=None if dr is None else dr.cuda())
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    alone, none = afd.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), weight_grad=False,
                                    grad_residual=None if dr is None else dr.cuda())
    assert none is None and torch.equal(alone, dh)


@pytest.mark.parametrize("T,H", [(4097, 2048), (2500, 4096), (3001, 264), (600, 16384), (1024, 2048), (1025, 2048), (512, 16384),
                                 (301, 40), (511, 4104), (900, 1504)])
@pytest.mark.parametrize("ht", [BF, F32])
def test_norm_grad_many_rows(T, H, ht):
    afd = _afd()
    _print("norm grad rows", T, H, ht)
    g = _gen(T)
    h, w, dy = _rand(g, T, H, dtype=ht), 1 + _rand(g, H, std=0.3), _rand(g, T, H, dtype=BF)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dh, dw = afd.rms_norm_grad(dy.cuda(), _gapped(h, 8), w.cuda(), rstd.cuda())
    want, tol, wantw, tolw = ref.norm_grad(dy.double(), h.double(), w.double(), rstd.double(), None)
    ref.check(dh, want, ref.rounded(want, tol, ht), "dh")
    ref.check(dw, wantw, tolw + ref.U * wantw.abs(), "dweight")


def test_norm_gradient_by_differences():
    """The gradients against differences of the 64-bit norm itself, not of a formula for them."""
    afd = _afd()
    g = _gen(17)
    T, H, step = 3, 64, 2.0 ** -10
    x, w, dy = _rand(g, T, H, std=1.5), 1 + _rand(g, H, std=0.3), _rand(g, T, H, dtype=BF)
    with torch.no_grad():
        n = afd.rms_norm(x.cuda(), w.cuda(), keep_rstd=True)
        dh, dw = (t.double().cpu() for t in afd.rms_norm_grad(dy.cuda(), x.cuda(), w.cuda(), n.rstd))
    d = dy.double()
    _, rstd, _, _ = ref.norm(x.double(), w, None, 1e-6)
    _, tol, _, tolw = ref.norm_grad(d, x.double(), w.double(), rstd, None)
    for i in range(H):
        e = torch.zeros(H, dtype=torch.float64)
        e[i] = step
        up, down = (ref.norm(x.double() + s * e, w, None, 1e-6)[2] for s in (1, -1))
        diff = ((up - down) * d).sum(1) / (2 * step)
        # |x_j| is at most sqrt(H) / rstd, so a third derivative at most 36 rstd^3 / H of the sum of sizes;
        # rstd moves by less than a factor 1.1 over the step; 4 roundings of the given rstd
        third = 36 * 1.1 ** 3 * rstd ** 3 / H * (d * w.double()).abs().sum(1)
        assert ((diff - dh[:, i]).abs() <= tol[:, i] + 4 * ref.U * dh[:, i].abs() + step ** 2 / 6 * third).all(), i
        up, down = (ref.norm(x.double(), w.double() + s * e, None, 1e-6)[2] for s in (1, -1))
        diff = ((up - down) * d).sum() / (2 * step)
        assert (diff - dw[i]).abs() <= tolw[i] + 8 * ref.U * (d * x.double() * rstd[:, None])[:, i].abs().sum(), i


def test_norm_grad_in_place_and_empty():
    """dh in place of either gradient, with few rows (where other workgroups read grad for dweight) and many."""
    afd = _afd()
    g = _gen(1)
    for T, H in ((33, 2048), (700, 4096), (1024, 512), (1500, 2048)):
        h, w, dy, dr = (_rand(g, *s, dtype=BF).cuda() for s in ((T, H), (H,), (T, H), (T, H)))
        rstd = torch.rand(T, generator=g).cuda() + 0.5
        want = afd.rms_norm_grad(dy, h, w, rstd, grad_residual=dr)
        for _ in range(5):
            a, b = dr.clone(), dy.clone()
            got = afd.rms_norm_grad(dy, h, w, rstd, grad_residual=a, out=a)
            assert got[0] is a and torch.equal(a, want[0]) and torch.equal(got[1], want[1])
            got = afd.rms_norm_grad(b, h, w, rstd, grad_residual=dr, out=b)
            assert got[0] is b and torch.equal(b, want[0]) and torch.equal(got[1], want[1])
    dh, dw = afd.rms_norm_grad(dy[:0], h[:0], w, rstd[:0])
    assert dh.shape == (0, 2048) and torch.equal(dw, torch.zeros(2048, device="cuda"))
    assert afd.rms_norm(h[:0], w).rows.shape == (0, 2048)


# ------------------------------------------------------------------ routes --

EXPERTS = [(1, 1), (2, 2), (5, 3), (8, 8), (40, 6), (63, 4), (64, 32), (65, 1), (96, 6), (128, 8), (128, 32), (130, 17),
           (256, 8), (257, 8), (384, 10), (511, 32), (512, 8)]


def _logits(g, T, E, dtype):
    l = _rand(g, T, E, std=1.5) + _rand(g, E)
    if dtype is BF:
        l = l.to(BF)
    return l


@pytest.mark.parametrize("E,K", EXPERTS)
@pytest.mark.parametrize("dtype,scoring,bias,renormalize,scale,T", [
    (F32, "softmax", False, True, 1.0, 37), (BF, "softmax", False, False, 2.5, 64), (F32, "sigmoid", True, True, 2.5, 50),
    (BF, "sigmoid", False, True, 1.0, 19), (F32, "sigmoid", False, False, -1.5, 1), (F32, "softmax", True, False, 1.0, 300),
    (BF, "softmax", True, True, 1.0, 3)])
def test_route(E, K, dtype, scoring, bias, renormalize, scale, T):
    afd = _afd()
    _print("route", E, K, dtype, scoring, bias, renormalize, T)
    g = _gen(E * 100 + K)
    logits, b = _logits(g, T, E, dtype), _rand(g, E, std=0.2) if bias else None
    live = torch.rand(T, generator=g) < 0.8
    for mask in (None, live):
        r = afd.route_tokens(logits.cuda(), K, scoring=scoring, bias=None if b is None else b.cuda(),
                             renormalize=renormalize, scale=scale, live=None if mask is None else mask.cuda())
        ids = ref.choose(logits, K, scoring, b, mask)
        assert r.ids.dtype is torch.int32 and torch.equal(r.ids.cpu().long(), ids)
        w, tol = ref.weights(logits, ids, scoring, renormalize, scale)
        ref.check(r.weights, w, tol, "weights")
        if mask is not None:
            assert (r.weights.cpu()[~mask] == 0).all()


@pytest.mark.parametrize("T,E,K", [(8193, 128, 8), (9000, 65, 17), (8200, 100, 32), (20001, 40, 3), (9001, 300, 6), (40000, 12, 2)])
@pytest.mark.parametrize("dtype,scoring,bias,renormalize", [(F32, "softmax", False, False), (BF, "sigmoid", True, True),
                                                            (F32, "sigmoid", True, False), (BF, "softmax", False, True)])
def test_route_many_rows(T, E, K, dtype, scoring, bias, renormalize):
    """More tokens than the forms for few take, and than the gradient's workgroups hold at once."""
    afd = _afd()
    _print("route rows", T, E, K, dtype, scoring, bias, renormalize)
    g = _gen(T + E)
    logits, b = _logits(g, T, E, dtype), _rand(g, E, std=0.2) if bias else None
    logits[7::11, ::2] = -INF
    r = afd.route_tokens(logits.cuda(), K, scoring=scoring, bias=None if b is None else b.cuda(), renormalize=renormalize)
    ids = ref.choose(logits, K, scoring, b, None)
    assert torch.equal(r.ids.cpu().long(), ids)
    ref.check(r.weights, *ref.weights(logits, ids, scoring, renormalize, 1.0), "weights")
    dw = _rand(g, T, K)
    d = afd.route_tokens_grad(dw.cuda(), logits.cuda(), r.ids, scoring=scoring, renormalize=renormalize)
    want, tol = ref.route_grad(dw, logits, ids, scoring, renormalize, 1.0)
    ref.check(d, want, ref.rounded(want, tol, dtype), "dlogits")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,K", [(8, 4), (128, 8), (256, 8), (500, 12)])
def test_route_odd_logits(scoring, dtype, biased, E, K):
    """Rows with ties, with infinities and NaNs, with masks that leave few experts or none, with the
    type's lowest value, and far from zero."""
    afd = _afd()
    _print("odd logits", scoring, dtype, biased, E, K)
    low = torch.finfo(dtype).min
    g = _gen(5)
    l = _logits(g, 16, E, dtype)
    l[0] = 0.0
    l[1] = -INF
    l[2] = NAN
    l[3] = low
    l[4] = -INF
    l[4, E // 2] = 1.0
    l[5, ::2] = -INF
    l[6, 1::3] = NAN
    l[7] = -INF
    l[7, :K - 1] = torch.arange(K - 1, dtype=F32).to(dtype)
    l[8] = low
    l[8, 3] = low / 2
    l[9, 2] = INF
    l[10, 1], l[10, E - 1] = INF, INF
    l[11] = l[11] - 300
    l[12] = l[12] + 300
    l[13] = (l[13] * 4).round() / 4
    l[14] = -INF
    l[14, :2] = low
    l[15] = l[15] * 40
    b = (_rand(g, E, std=0.2) * 8).round() / 8 if biased else None
    if biased:
        b[0], b[5 % E], b[6 % E] = -INF, NAN, INF
    for renormalize in (True, False):
        r = afd.route_tokens(l.cuda(), K, scoring=scoring, bias=None if b is None else b.cuda(), renormalize=renormalize)
        ids = ref.choose(l, K, scoring, b, None)
        keep = torch.ones(16, dtype=torch.bool)
        if biased:
            # scores that differ by less than 64-bit exponentials are off may change places: rows far
            # from zero, where many sigmoids are within a few steps of 1
            keep[[12, 15]] = False
        assert torch.equal(r.ids.cpu().long()[keep], ids[keep])
        ids = r.ids.cpu().long()
        w, tol = ref.weights(l, ids, scoring, renormalize, 1.0)
        ref.check(r.weights, w, tol, "weights")
        s = r.weights.cpu().double()
        assert not s.isnan().any() and (s[ids < 0] == 0).all()
        if renormalize:
            full = (ids >= 0).any(1)
            assert ((s.sum(1)[full] - 1).abs() < 64 * 2 ** -24).all()
        for row in ids.tolist():
            chosen = [i for i in row if i >= 0]
            assert len(set(chosen)) == len(chosen) and all(i < E for i in chosen)
            assert row == chosen + [-1] * (K - len(chosen))


@pytest.mark.parametrize("E,gap,off", [(128, 3, 0), (128, 0, 1), (96, 4, 2), (96, 32, 0), (250, 6, 0), (300, 1, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_of_any_stride(E, gap, off, dtype):
    afd = _afd()
    _print("strides", E, gap, off, dtype)
    g = _gen(2)
    l, K, T = _logits(g, 40, E, dtype), 6, 40
    buf = torch.full((T * (E + gap) + off + 8,), NAN, dtype=dtype, device="cuda")
    v = buf[off:off + T * (E + gap)].view(T, E + gap)[:, :E]
    v.copy_(l)
    dw, gl = _rand(g, T, K).cuda(), torch.tensor(0.7, device="cuda")
    a, b = (afd.route_tokens(t, K, renormalize=False) for t in (l.cuda(), v))
    assert torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)
    x, y = (afd.route_tokens_grad(dw, t, a.ids, renormalize=False) for t in (l.cuda(), v))
    assert torch.equal(x, y)
    p, q = (afd.balance_loss(t, a.ids) for t in (l.cuda(), v))
    assert all(torch.equal(i, j) for i, j in zip(p, q))
    x, y = (afd.balance_loss_grad(gl, t, a.ids, p.slope) for t in (l.cuda(), v))
    assert torch.equal(x, y)
    if not off:      # a gradient that is not aligned for wide stores
        out = torch.empty(T * E + 1, dtype=dtype, device="cuda")[1:].view(T, E)
        assert torch.equal(afd.balance_loss_grad(gl, v, a.ids, p.slope, out=out), x)


@pytest.mark.parametrize("E,K", EXPERTS)
@pytest.mark.parametrize("dtype,scoring,renormalize,scale,T", [
    (F32, "softmax", False, 1.0, 37), (BF, "softmax", True, 2.5, 50), (F32, "sigmoid", True, 2.5, 64),
    (F32, "sigmoid", False, 1.0, 3), (F32, "softmax", True, 1.0, 1)])
def test_route_grad(E, K, dtype, scoring, renormalize, scale, T):
    afd = _afd()
    _print("route grad", E, K, dtype, scoring, renormalize, T)
    g = _gen(E * 100 + K)
    logits, dw = _logits(g, T, E, dtype), _rand(g, T, K)
    live = torch.rand(T, generator=g) < 0.8
    ids = ref.choose(logits, K, scoring, None, live)
    dw[~live] = NAN                                  # of weights that are not there
    d = afd.route_tokens_grad(dw.cuda(), logits.cuda(), ids.int().cuda(), scoring=scoring, renormalize=renormalize,
                              scale=scale)
    want, tol = ref.route_grad(dw, logits, ids, scoring, renormalize, scale)
    ref.check(d, want, ref.rounded(want, tol, dtype), "dlogits")
    assert (d.cpu()[~live] == 0).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_grad_odd(scoring, renormalize):
    """Masked logits, the same id twice, ids out of range, and logits far from zero."""
    afd = _afd()
    g = _gen(9)
    T, E, K = 8, 100, 5
    l = _rand(g, T, E)
    l[0] = -INF
    l[1, ::2] = -INF
    l[2, 4], l[2, 8] = NAN, -INF
    l[4] -= 250
    l[5] += 250
    l[6] = torch.finfo(F32).min
    ids = ref.choose(l, K, scoring, None, None)
    ids[2, :2] = torch.tensor([4, 8])                # experts that cannot be chosen
    ids[3] = torch.tensor([7, 7, 9, 7, -1])
    ids[7] = torch.tensor([100, -5, 2 ** 30, 3, -2 ** 31])
    dw = _rand(g, T, K)
    d = afd.route_tokens_grad(dw.cuda(), l.cuda(), ids.int().cuda(), scoring=scoring, renormalize=renormalize)
    want, tol = ref.route_grad(dw, l, ids, scoring, renormalize, 1.0)
    ref.check(d, want, ref.rounded(want, tol, F32), "dlogits")


def test_route_gradient_by_differences():
    """The gradient against differences of the call's own weights, whose error is theirs over the step."""
    afd = _afd()
    g = _gen(4)
    T, E, K, step = 6, 24, 4, 2.0 ** -6
    l = torch.stack([torch.randperm(E, generator=g).float() / 2 for _ in range(T)])     # gaps of 1/2: the choice stands
    dw = _rand(g, T, K)
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            kw = dict(scoring=scoring, renormalize=renormalize, scale=1.5)
            r = afd.route_tokens(l.cuda(), K, **kw)
            d = afd.route_tokens_grad(dw.cuda(), l.cuda(), r.ids, **kw).double().cpu()
            for e in range(E):
                side = []
                for s in (step, -step):
                    x = l.clone()
                    x[:, e] += s
                    q = afd.route_tokens(x.cuda(), K, **kw)
                    assert torch.equal(q.ids, r.ids)
                    side.append((q.weights.double().cpu() * dw.double()).sum(1))
                diff = (side[0] - side[1]) / (2 * step)
                # third derivatives of a softmax or sigmoid are at most 1 in size: step^2 / 6 each
                size = dw.double().abs().sum(1) * 1.5
                tol = size * (step ** 2 / 6 + 200 * ref.U / step)
                assert ((diff - d[:, e]).abs() <= tol).all(), (scoring, renormalize, e)


# ------------------------------------------------------------ balance loss --

@pytest.mark.parametrize("E,K", EXPERTS)
@pytest.mark.parametrize("dtype,scoring,T,coefficient", [(F32, "softmax", 37, 1.0), (BF, "softmax", 300, 0.01),
                                                         (F32, "sigmoid", 1, 1.0), (BF, "sigmoid", 70, -2.0)])
def test_balance(E, K, dtype, scoring, T, coefficient):
    afd = _afd()
    _print("balance", E, K, dtype, scoring, T)
    g = _gen(E * 100 + K + 1)
    logits = _logits(g, T, E, dtype)
    live = torch.rand(T, generator=g) < 0.8
    for mask in (None, live):
        ids = ref.choose(logits, K, scoring, None, mask)
        _check_balance(afd, logits, ids, scoring, coefficient)


def _check_balance(afd, logits, ids, scoring, coefficient):
    b = afd.balance_loss(logits.cuda(), ids.int().cuda(), scoring=scoring, coefficient=coefficient)
    loss, tol, counts, slope, p, on = ref.balance(logits, ids, scoring, coefficient)
    assert b.counts.dtype is torch.int32 and torch.equal(b.counts.cpu().long(), counts)
    ref.check(b.slope, slope, 2 * ref.U * slope.abs(), "slope")
    ref.check(b.loss, loss, tol, "loss")
    grad = torch.tensor(0.75)
    d = afd.balance_loss_grad(grad.cuda(), logits.cuda(), ids.int().cuda(), b.slope, scoring=scoring)
    want, tol = ref.balance_grad(0.75, logits, p, b.slope.double().cpu(), on, scoring)
    ref.check(d, want, ref.rounded(want, tol, logits.dtype), "dlogits")
    assert (d.cpu()[~on] == 0).all()
    again = afd.balance_loss(logits.cuda(), ids.int().cuda(), scoring=scoring, coefficient=coefficient)
    assert all(torch.equal(x, y) for x, y in zip(b, again))
    return b


@pytest.mark.parametrize("T,E,K", [(5000, 96, 6), (9001, 128, 8), (4097, 512, 8), (70000, 16, 2), (5000, 200, 8),
                                   (20000, 300, 4)])
def test_balance_many_rows(T, E, K):
    afd = _afd()
    _print("balance rows", T, E, K)
    g = _gen(T)
    logits = _logits(g, T, E, F32)
    _check_balance(afd, logits, ref.choose(logits, K, "softmax", None, torch.rand(T, generator=g) < 0.9), "softmax", 0.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_odd(scoring):
    """No token, no counting token, masked experts, repeated ids and ids out of range, logits far from zero."""
    afd = _afd()
    g = _gen(11)
    E, K = 96, 6
    l = _rand(g, 12, E)
    l[0] = -INF
    l[1, ::2] = -INF
    l[2, 3], l[2, 5] = NAN, -INF
    l[3] -= 300
    l[4] += 300
    l[5] = torch.finfo(F32).min
    l[6, 7] = INF
    ids = ref.choose(l, K, scoring, None, None)
    ids[0, 0] = 3                                    # a token without an expert that counts all the same
    ids[7] = 9
    ids[8] = torch.tensor([96, -3, 2 ** 30, -2 ** 31, 512, -1])
    ids[9] = torch.tensor([-1, -1, 4, -1, -1, -1])
    _check_balance(afd, l, ids, scoring, 1.0)
    none = torch.full((12, K), -1)
    b = _check_balance(afd, l, none, scoring, 1.0)
    assert float(b.loss) == 0 and int(b.counts.sum()) == 0
    b = afd.balance_loss(l[:0].cuda(), none[:0].int().cuda(), scoring=scoring)
    assert float(b.loss) == 0 and (b.counts == 0).all() and (b.slope == 0).all()
    assert afd.balance_loss_grad(torch.ones((), device="cuda"), l[:0].cuda(), none[:0].int().cuda(), b.slope).shape == (0, E)


def test_balance_of_even_use_is_the_coefficient():
    afd = _afd()
    for E, K in ((8, 2), (128, 8), (512, 4)):
        ids = torch.arange(E * K).reshape(E, K) % E
        b = afd.balance_loss(torch.zeros(E, E).cuda(), ids.int().cuda(), coefficient=0.25)
        assert abs(float(b.loss) - 0.25) < 0.25 * 64 * ref.U and (b.counts == K).all()


def test_balance_gradient_by_differences():
    afd = _afd()
    g = _gen(6)
    T, E, K, step = 5, 24, 4, 2.0 ** -6
    for scoring in ("softmax", "sigmoid"):
        l = _rand(g, T, E)
        ids = ref.choose(l, K, scoring, None, None).int().cuda()
        b = afd.balance_loss(l.cuda(), ids, scoring=scoring)
        d = afd.balance_loss_grad(torch.ones((), device="cuda"), l.cuda(), ids, b.slope, scoring=scoring).double().cpu()
        size = float(b.slope.abs().max())
        for t in range(T):
            for e in range(E):
                side = []
                for s in (step, -step):
                    x = l.clone()
                    x[t, e] += s
                    side.append(float(afd.balance_loss(x.cuda(), ids, scoring=scoring).loss))
                # third derivatives of shares are at most 2 in size, one token's shares sum to 1
                assert abs((side[0] - side[1]) / (2 * step) - d[t, e]) <= size * (step ** 2 / 3 + 100 * T * ref.U / step)


# ------------------------------------------------- autograd, streams, graphs --

def test_autograd():
    """backward() through the three calls against their own gradient calls."""
    afd = _afd()
    g = _gen(3)
    T, H, E, K = 50, 512, 64, 4
    x, r, w = (_rand(g, *s, dtype=t).cuda().requires_grad_() for s, t in (((T, H), BF), ((T, H), F32), ((H,), BF)))
    l = _rand(g, T, E).cuda().requires_grad_()
    n = afd.rms_norm(x, w, r)
    gy, gh = _rand(g, T, H, dtype=BF).cuda(), _rand(g, T, H).cuda()
    torch.autograd.backward([n.rows, n.residual], [gy, gh])
    with torch.no_grad():
        m = afd.rms_norm(x, w, r, keep_rstd=True)
        dh, dw = afd.rms_norm_grad(gy, m.residual, w, m.rstd, grad_residual=gh)
    assert torch.equal(r.grad, dh) and torch.equal(x.grad, dh.to(BF)) and torch.equal(w.grad, dw.to(BF))
    routes = afd.route_tokens(l, K, scale=2.0)
    b = afd.balance_loss(l, routes.ids, coefficient=0.1)
    gw = _rand(g, T, K).cuda()
    ((routes.weights * gw).sum() + b.loss * 3).backward()
    with torch.no_grad():
        want = afd.route_tokens_grad(gw, l, routes.ids, scale=2.0) + \
            afd.balance_loss_grad(torch.tensor(3.0, device="cuda"), l, routes.ids, b.slope)
    assert torch.equal(l.grad, want)
    # only the rows, only the stream, only the weight; expanded gradients
    for rows, stream in ((True, False), (False, True)):
        x.grad = r.grad = w.grad = None
        n = afd.rms_norm(x, w, r)
        (n.rows if rows else n.residual).sum().backward()
        assert x.grad is not None and r.grad is not None and (w.grad is not None) == rows
    n = afd.rms_norm(x.detach(), w, r.detach())
    assert n.rows.requires_grad and not n.residual.requires_grad
    w.grad = None
    n.rows.float().sum().backward()
    assert w.grad.shape == (H,)
    same = _rand(g, T, H, dtype=BF).cuda().requires_grad_()
    afd.rms_norm(same, w.detach(), same).rows.sum().backward()         # x and the residual are one tensor
    with torch.no_grad():
        m = afd.rms_norm(same, w, same, keep_rstd=True)
        dh, _ = afd.rms_norm_grad(torch.ones_like(m.rows), m.residual, w, m.rstd)
    assert torch.equal(same.grad, dh + dh)
    y = afd.rms_norm(same, w)                                           # without a residual
    (g1,) = torch.autograd.grad(y.rows, same, torch.ones_like(y.rows))
    with torch.no_grad():
        m = afd.rms_norm(same, w, keep_rstd=True)
        assert torch.equal(g1, afd.rms_norm_grad(torch.ones_like(m.rows), same, w, m.rstd)[0])


def test_autograd_refusals():
    afd = _afd()
    x, w = torch.randn(4, 256, device="cuda", dtype=BF, requires_grad=True), torch.ones(256, device="cuda", dtype=BF)
    l = torch.randn(4, 8, device="cuda", requires_grad=True)
    for kw in (dict(dtype=F8), dict(out=torch.empty_like(w.expand(4, 256).contiguous()))):
        with pytest.raises(ValueError, match="gradient"):
            afd.rms_norm(x, w, **kw)
    with pytest.raises(ValueError, match="gradient"):
        afd.route_tokens(l, 2, ids=torch.empty(4, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="gradient"):
        afd.route_tokens(l.detach(), 2, bias=torch.zeros(8, device="cuda", requires_grad=True))
    with pytest.raises(ValueError, match="gradient"):
        afd.balance_loss_grad(torch.ones((), device="cuda"), l, torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                              torch.ones(8, device="cuda"))
    out = afd.rms_norm(x, w).rows
    (once,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        once.sum().backward()                        # no second derivative
    # a capture records no autograd graph; its gradient calls are there instead
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        try:
            with pytest.raises(ValueError, match="captured"):
                afd.rms_norm(x, w)
            with pytest.raises(ValueError, match="captured"):
                afd.route_tokens(l, 2)
            with torch.no_grad():
                afd.rms_norm(x, w)
        finally:
            graph.capture_end()
    torch.cuda.current_stream().wait_stream(stream)


def test_graph_replays():
    """A training step's calls captured twice, replayed in turns with inputs that change in place, eager work
    between them."""
    afd = _afd()
    g = _gen(8)
    T, H, E, K = 96, 1024, 96, 6

    def inputs():
        return [_rand(g, T, H, dtype=BF).cuda(), _rand(g, T, H, dtype=BF).cuda(), _rand(g, T, E).cuda(),
                _rand(g, T, H, dtype=BF).cuda(), _rand(g, T, K).cuda()]

    w, one = (1 + _rand(g, H, std=0.2)).cuda(), torch.ones((), device="cuda")

    def step(x, r, l, gy, gw):
        n = afd.rms_norm(x, w, r, keep_rstd=True)
        f = afd.rms_norm(x, w, dtype=F8)
        t = afd.route_tokens(l, K)
        b = afd.balance_loss(l, t.ids)
        return [n.rows, n.residual, n.rstd, f.rows, f.scales, t.ids, t.weights, *b,
                *afd.rms_norm_grad(gy, n.residual, w, n.rstd, grad_residual=x),
                afd.route_tokens_grad(gw, l, t.ids), afd.balance_loss_grad(one, l, t.ids, b.slope)]

    held = [inputs(), inputs()]
    for h in held:
        step(*h)
    torch.cuda.synchronize()
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    for h in held:                                   # both from one pool
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(step(*h))
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1):
            for t, n in zip(held[i], inputs()):
                t.copy_(n)
            graphs[i].replay()
            got = [o.clone() for o in outs[i]]
            torch.cuda.synchronize()
            want = step(*held[i])
            for k, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a.float() if a.element_size() == 1 else a, b.float() if b.element_size() == 1 else b), \
                    (turn, i, k)


def test_side_streams():
    """Two streams at once, on inputs made on another."""
    afd = _afd()
    g = _gen(12)
    T, H, E, K = 300, 2048, 128, 8
    x, w, l, gy = _rand(g, T, H, dtype=BF).cuda(), torch.ones(H, device="cuda"), _rand(g, T, E).cuda(), \
        _rand(g, T, H, dtype=BF).cuda()

    def step():
        n = afd.rms_norm(x, w, keep_rstd=True)
        t = afd.route_tokens(l, K)
        return [n.rows, t.ids, t.weights, *afd.balance_loss(l, t.ids), *afd.rms_norm_grad(gy, x, w, n.rstd)]

    want = step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    for s in streams:
        s.synchronize()
    for outs in got:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


# --------------------------------------------------------------- one round --

@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_rounds_of_two_layers(dtype):
    """Two layers as a source runs them: norm with the residual, logits, routes, dispatch, experts, reply,
    collect, and the next layer's norm; against the same round fed by the plain calls."""
    afd = _afd()
    from tests import experts_ref as er
    N, F, E, K, H, I, alpha, T = 2, 2, 8, 2, 512, 256, 16, 24
    g = _gen(21)
    fp8 = dtype == "fp8"
    dev = lambda t: None if t is None else t.view(torch.uint8).cuda().view(t.dtype) if t.element_size() == 1 else t.cuda()  # noqa: E731
    buf = afd.Buffer(N, F, E, K, H, alpha, T, dtype=dtype)
    experts = []
    for f in range(F):
        up = er.make(31 + f, E // F, [1] * (E // F), 1, H, 2 * I, dtype, gated=True)
        down = er.make(41 + f, E // F, [1] * (E // F), 1, I, H, dtype)
        experts.append(afd.Experts(dev(up["w"]), dev(down["w"]), dev(up["ws"]), dev(down["ws"])))
    w, gate = (1 + _rand(g, H, std=0.2)).cuda(), _rand(g, E, H, std=H ** -0.5).cuda()
    live = torch.ones(T, dtype=torch.bool)
    live[5], live[T - 1] = False, False
    live = live.cuda()
    stream = [_rand(g, T, H, dtype=BF).cuda() for _ in range(N)]
    x = [_rand(g, T, H, dtype=BF).cuda() for _ in range(N)]
    for layer in range(2):
        sent = []
        for s in range(N):
            n = buf.source_norm(s, x[s], w, stream[s], residual_out=stream[s])
            logits = afd.rms_norm(stream[s], w).rows.float() @ gate.t()
            r = buf.source_route(s, logits, live=live)
            buf.source_dispatch(s, n.rows, r.ids, r.weights, n.scales, bucket=T)
            sent.append((n, r))
        recs = [buf.worker_receive(f, bucket=T) for f in range(F)]
        for f, rec in enumerate(recs):
            buf.worker_reply(f, buf.worker_experts(f, rec, experts[f]), rec.receipt)
        x = [buf.source_collect(s).clone() for s in range(N)]
        assert buf.get_error() == (0, -1, -1, -1)
        for s, (n, r) in enumerate(sent):
            assert (x[s][~live] == 0).all() and (r.ids[~live] == -1).all() and (x[s][live] != 0).any()
            # every token again: its experts' network applied to its row alone, weighted
            tot = torch.zeros(T, H, device="cuda")
            for k in range(K):
                for e in range(E):
                    at = torch.nonzero(r.ids[:, k] == e).reshape(-1)
                    if not len(at):
                        continue
                    ends = torch.zeros(E // F, dtype=torch.int32)
                    ends[e % (E // F):] = len(at)
                    rows = n.rows[at] if not fp8 else n.rows.view(torch.uint8)[at].view(F8)
                    y = afd.expert_ffn(rows.contiguous(), ends.cuda(), experts[e // (E // F)],
                                       x_scales=n.scales[at].contiguous() if fp8 else None)
                    tot[at] += r.weights[at, k:k + 1] * y.float()
            # the round's experts and these may take different kernels: rows equal to a BF16 step, and one more for the sum
            size = tot.abs().amax(1, keepdim=True)
            assert ((x[s].float() - tot).abs() <= size * 2.0 ** -6).all(), (layer, s)


# ------------------------------------------------ borders, sizes, refusals --

@pytest.mark.parametrize("E,K", [(40, 6), (128, 8), (200, 9), (256, 32), (300, 8), (512, 8), (512, 32)])
@pytest.mark.parametrize("levels", [1, 2, 4, 30, 200])
@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_ties(E, K, levels, scoring, biased):
    """Logits of a few levels: many equal ones at every border, all of them where there is one level."""
    afd = _afd()
    _print("ties", E, K, levels, scoring, biased)
    g = _gen(E + levels)
    for dtype in (F32, BF):
        l = (torch.randint(0, levels, (40, E), generator=g) / 64).to(dtype)
        l[::5, ::3] = -INF
        b = torch.randint(0, 3, (E,), generator=g) / 4 if biased else None
        r = afd.route_tokens(l.cuda(), K, scoring=scoring, bias=None if b is None else b.cuda())
        ids = r.ids.cpu().long()
        want = ref.choose(l, K, scoring, b, None)
        if b is None:
            assert torch.equal(ids, want)
        else:
            # equal logits have equal scores whatever computes them; different ones with different biases may
            # come within a 64-bit exponential's error of each other, or not: the keys have to agree
            key = torch.where(ref.clean(l) == -INF, -INF, ref.scores(l, scoring) + b.double())
            a, c = (torch.take_along_dim(key, i.clamp(min=0), 1) for i in (ids, want))
            assert torch.equal(ids < 0, want < 0) and ((a - c).abs()[want >= 0] <= 2.0 ** -50).all()
            same = (ids == want) | ((a - c).abs() <= 2.0 ** -50) & (a != c)
            assert same.all() or torch.equal(a, c) and torch.equal(ids, want)


@pytest.mark.parametrize("E,K", [(16, 4), (128, 8), (256, 8), (512, 8), (512, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_scores_nearer_than_float32(E, K, scoring):
    """Neighbouring float32 logits: scores that float32 cannot tell apart, 64 bits can."""
    afd = _afd()
    g = _gen(E)
    base = torch.full((), 2.0) if scoring == "sigmoid" else torch.full((), 1.0)
    step = torch.finfo(F32).eps * float(base)
    l = torch.stack([base + step * torch.randperm(E, generator=g) for _ in range(50)]).float()
    l[::2, E // 2:] = -1.0                          # fewer of them: settled among the picked
    l[::7, 12:] = -1.0
    b = torch.zeros(E)
    r = afd.route_tokens(l.cuda(), K, scoring=scoring, bias=b.cuda())
    assert torch.equal(r.ids.cpu().long(), ref.choose(l, K, scoring, b, None))


def test_norm_of_more_rows_than_a_launch():
    afd = _afd()
    T, H = (1 << 20) + 5, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.randn(T, H, generator=g, device="cuda").to(BF), torch.rand(H, generator=g, device="cuda")
    n = afd.rms_norm(x, w, x, keep_rstd=True)
    for at in (0, (1 << 20) - 3, T - 4):
        s = slice(at, at + 4)
        m = afd.rms_norm(x[s], w, x[s], keep_rstd=True)
        assert all(a is None or torch.equal(a[s], b) for a, b in zip(n, m))


def test_offsets_past_32_bits():
    afd = _afd()
    T, H = 140001, 16384                            # 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    _print("offsets", T, H)
    x = torch.empty(T, H, dtype=BF, device="cuda")
    x[:1000] = torch.randn(1000, H, generator=g, device="cuda").to(BF)
    x[1000:] = 0.5
    x[-50:] = torch.randn(50, H, generator=g, device="cuda").to(BF)
    w, tail = torch.rand(H, generator=g, device="cuda"), slice(T - 50, T)
    n = afd.rms_norm(x, w, x, keep_rstd=True)
    m = afd.rms_norm(x[tail].clone(), w, x[tail].clone(), keep_rstd=True)
    assert all(a is None or torch.equal(a[tail], b) for a, b in zip(n, m))
    f = afd.rms_norm(x, w, dtype=F8, out=torch.empty(T, H, dtype=F8, device="cuda"))
    q = afd.rms_norm(x[tail].clone(), w, dtype=F8)
    assert torch.equal(f.rows[tail].view(torch.uint8), q.rows.view(torch.uint8)) and torch.equal(f.scales[tail], q.scales)
    del f
    d, _ = afd.rms_norm_grad(n.rows, n.residual, w, n.rstd, out=x)
    e, _ = afd.rms_norm_grad(m.rows, m.residual, w, m.rstd)
    assert torch.equal(d[tail], e)
    del d, n, x
    T, E, K = (1 << 22) + 1001, 512, 8
    l = torch.zeros(T, E, device="cuda")
    l[-50:] = torch.randn(50, E, generator=g, device="cuda")
    tail = slice(T - 50, T)
    r = afd.route_tokens(l, K, renormalize=False)
    t = l[tail].clone()
    s = afd.route_tokens(t, K, renormalize=False)
    assert torch.equal(r.ids[tail], s.ids) and torch.equal(r.weights[tail], s.weights)
    assert torch.equal(r.ids[0].cpu(), torch.arange(K, dtype=torch.int32))
    dw = torch.ones(T, K, device="cuda")
    dw[-50:] = torch.randn(50, K, generator=g, device="cuda")
    d = afd.route_tokens_grad(dw, l, r.ids, renormalize=False)
    assert torch.equal(d[tail], afd.route_tokens_grad(dw[tail].clone(), t, s.ids, renormalize=False))
    b = afd.balance_loss(l, r.ids)
    assert int(b.counts.sum()) == T * K and int(b.counts[0]) >= T - 50
    one = torch.ones((), device="cuda")
    afd.balance_loss_grad(one, l, r.ids, b.slope, out=d)
    assert torch.equal(d[tail], afd.balance_loss_grad(one, t, s.ids, b.slope))


def test_refusals():
    afd = _afd()
    z = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    x, w, l, ids = z(4, 256, t=BF), z(256, t=BF), z(4, 8), z(4, 2, t=torch.int32)
    flat = z(4 * 264 + 8, t=BF)
    for call in (
            lambda: afd.rms_norm(x[0], w), lambda: afd.rms_norm(x.t(), w), lambda: afd.rms_norm(x[:, ::2], w[:128].contiguous()),
            lambda: afd.rms_norm(x, w[:128]), lambda: afd.rms_norm(x, w, x[:3]), lambda: afd.rms_norm(x, w, eps=0.0),
            lambda: afd.rms_norm(x, w, eps=float("nan")), lambda: afd.rms_norm(z(4, 252, t=BF), w[:252]),
            lambda: afd.rms_norm(z(4, 136, t=BF), w[:136], dtype=F8), lambda: afd.rms_norm(z(2, 16392, t=BF), z(16392)),
            lambda: afd.rms_norm(x, w, out=z(4, 256)), lambda: afd.rms_norm(x, w, out=z(3, 256, t=BF)),
            lambda: afd.rms_norm(x, w, out_scales=z(4, 2)), lambda: afd.rms_norm(x, w, residual_out=x),
            lambda: afd.rms_norm(x, w, x, residual_out=z(4, 256)), lambda: afd.rms_norm(x, w, dtype=F8, out_scales=z(4, 1)),
            lambda: afd.rms_norm(flat[1:1025].view(4, 256), w), lambda: afd.rms_norm(x, flat[1:257]),
            lambda: afd.rms_norm(flat[:4 * 260].view(4, 260)[:, :256], w), lambda: afd.rms_norm(x[:1].expand(4, 256), w),
            lambda: afd.rms_norm(x, w.cpu()), lambda: afd.rms_norm(x, w, x.cpu()),
            lambda: afd.rms_norm_grad(x[:3], x, w, z(4)), lambda: afd.rms_norm_grad(x, x, w, z(3)),
            lambda: afd.rms_norm_grad(x.float(), x, w, z(4)), lambda: afd.rms_norm_grad(x, x, w, z(4), grad_residual=z(4, 256)),
            lambda: afd.rms_norm_grad(x, x, w, z(4), out=z(4, 256)),
            lambda: afd.route_tokens(l, 0), lambda: afd.route_tokens(l, 9), lambda: afd.route_tokens(l[0], 2),
            lambda: afd.route_tokens(l.t(), 2), lambda: afd.route_tokens(z(2, 513), 2), lambda: afd.route_tokens(z(2, 0), 1),
            lambda: afd.route_tokens(l, 2, scoring="tanh"), lambda: afd.route_tokens(l, 2, scale=float("inf")),
            lambda: afd.route_tokens(l, 2, bias=z(7)), lambda: afd.route_tokens(l, 2, bias=z(8, t=BF)),
            lambda: afd.route_tokens(l, 2, live=z(4)), lambda: afd.route_tokens(l, 2, live=z(3, t=torch.bool)),
            lambda: afd.route_tokens(l, 2, ids=z(4, 2)), lambda: afd.route_tokens(l, 2, weights=z(4, 3)),
            lambda: afd.route_tokens(l[:1].expand(4, 8), 2),
            lambda: afd.route_tokens_grad(z(4, 2), l, ids.long()), lambda: afd.route_tokens_grad(z(4, 3), l, ids),
            lambda: afd.route_tokens_grad(z(4, 2), l, ids, out=z(4, 9)), lambda: afd.route_tokens_grad(z(4, 2), l, ids[:, 0]),
            lambda: afd.balance_loss(l, ids[:3]), lambda: afd.balance_loss(l, ids, coefficient=float("nan")),
            lambda: afd.balance_loss(l, z(4, 33, t=torch.int32)), lambda: afd.balance_loss_grad(z(1), l, ids, z(8)),
            lambda: afd.balance_loss_grad(z(), l, ids, z(7)), lambda: afd.balance_loss_grad(torch.zeros(()), l, ids, z(8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: afd.rms_norm(x.half(), w), lambda: afd.rms_norm(x, w.half()), lambda: afd.rms_norm(x, w, x.half()),
                 lambda: afd.rms_norm(x, w, dtype=torch.float16), lambda: afd.route_tokens(l.double(), 2),
                 lambda: afd.route_tokens(l, 2.5), lambda: afd.balance_loss(l.half(), ids)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: afd.rms_norm(x, w, x, out=x, residual_out=x), lambda: afd.rms_norm(x, w, out=w.expand(1, 256)),
                 lambda: afd.rms_norm_grad(x, x, w, z(4), out=x)):
        with pytest.raises((ValueError, afd.AfdError)):
            call()
    buf = afd.Buffer(1, 1, 8, 2, 256, capacity=4)
    for call in (lambda: buf.source_norm(1, x, w), lambda: buf.source_norm(0, z(5, 256, t=BF), w),
                 lambda: buf.source_norm(0, z(4, 128, t=BF), w[:128]), lambda: buf.source_route(0, z(4, 9)),
                 lambda: buf.source_route(-1, l), lambda: buf.source_route(0, l.cpu())):
        with pytest.raises(ValueError):
            call()
    asks = lambda t: t.clone().requires_grad_()  # noqa: E731
    for call in (lambda: buf.source_norm(0, asks(x), w), lambda: buf.source_norm(0, x, asks(w)),
                 lambda: buf.source_norm(0, x, w, asks(x)), lambda: buf.source_route(0, asks(l)),
                 lambda: buf.source_route(0, l, bias=asks(z(8)))):
        with pytest.raises(ValueError, match="no gradients"):
            call()
    with torch.no_grad():
        assert not buf.source_route(0, asks(l)).weights.requires_grad
    assert buf.source_norm(0, x, w).rows.shape == (4, 256) and buf.source_route(0, l).ids.shape == (4, 2)
