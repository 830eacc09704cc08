"""Host checks of the source's side (over the recording backend): refusals,
workspace sizes and the launches they lead to.  Refused calls launch nothing."""
import ctypes

import pytest

from combine_layout_amd import _native as nat
from tests.test_experts_host import log

BF16, FP8, FP32, NONE = nat.AFD_BF16, nat.AFD_FP8_E4M3, nat.AFD_FP32, nat.NO_RESIDUAL
X, R, W, OUT, OUTS, RO, RSTD, WS, DW = (i << 40 for i in range(1, 10))
ROWS = (1 << 24) - 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return nat.load_fake()


def ncfg(**kw):
    c = dict(hidden=256, x_dtype=BF16, residual_dtype=BF16, weight_dtype=BF16, out_dtype=BF16, eps=1e-6)
    c.update(kw)
    return nat.NormConfig(**c)


def norm(lib, c, rows=100, **kw):
    res, f8 = c.residual_dtype != NONE, c.out_dtype == FP8
    a = dict(x=X, xs=c.hidden, r=R if res else None, rs=c.hidden if res else 0, w=W, out=OUT, outs=OUTS if f8 else None,
             ro=RO if res else None, hs=c.hidden if res else 0, rstd=None)
    a.update(kw)
    return lib.afd_norm(ctypes.byref(c), rows, a["x"], a["xs"], a["r"], a["rs"], a["w"], a["out"], a["outs"], a["ro"], a["hs"],
                        a["rstd"], None)


def grad(lib, c, rows=100, **kw):
    a = dict(g=X, gr=R, h=OUT, hs=c.hidden, w=W, rstd=RSTD, dh=RO, dw=DW, ws=WS, wsb=1 << 40)
    a.update(kw)
    return lib.afd_norm_grad(ctypes.byref(c), rows, a["g"], a["gr"], a["h"], a["hs"], a["w"], a["rstd"], a["dh"], a["dw"],
                             a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(), dict(hidden=8), dict(hidden=16384), dict(out_dtype=FP8), dict(out_dtype=FP8, hidden=128),
                                dict(x_dtype=FP32), dict(residual_dtype=FP32), dict(residual_dtype=NONE),
                                dict(weight_dtype=FP32), dict(eps=1.17549435e-38), dict(eps=3e38)])
def test_norm_accepted(lib, kw):
    log(lib)
    c = ncfg(**kw)
    for rows in (1, 100, ROWS):
        assert norm(lib, c, rows, rstd=RSTD) == 0
        line, = log(lib)
        assert line.startswith(f"norm H={c.hidden} x32={int(c.x_dtype == FP32)} res={int(c.residual_dtype != NONE)} "
                               f"r32={int(c.residual_dtype == FP32)} w32={int(c.weight_dtype == FP32)} "
                               f"out8={int(c.out_dtype == FP8)} rows={rows} ")
        assert f"rstd={hex(RSTD)}" in line


@pytest.mark.parametrize("kw", [
    dict(hidden=0), dict(hidden=-8), dict(hidden=4), dict(hidden=12), dict(hidden=16392), dict(hidden=136, out_dtype=FP8),
    dict(x_dtype=FP8), dict(x_dtype=3), dict(x_dtype=-1), dict(residual_dtype=FP8), dict(residual_dtype=-2),
    dict(weight_dtype=FP8), dict(weight_dtype=-1), dict(out_dtype=FP32), dict(out_dtype=-1), dict(eps=0.0), dict(eps=-1e-6),
    dict(eps=1e-39), dict(eps=NAN), dict(eps=INF)])
def test_norm_shapes_refused(lib, kw):
    log(lib)
    need = ctypes.c_size_t()
    assert norm(lib, ncfg(**kw)) == nat.AFD_E_SHAPE
    assert grad(lib, ncfg(**kw)) == nat.AFD_E_SHAPE
    assert lib.afd_norm_grad_query(ctypes.byref(ncfg(**kw)), 5, ctypes.byref(need)) == nat.AFD_E_SHAPE
    assert log(lib) == []


@pytest.mark.parametrize("cfg,args", [
    ({}, dict(rows=-1)), ({}, dict(rows=1 << 24)), ({}, dict(x=None)), ({}, dict(x=X + 8)), ({}, dict(xs=248)),
    ({}, dict(xs=260)), ({}, dict(xs=1 << 31)), ({}, dict(xs=-256)), ({}, dict(r=None)), ({}, dict(r=R + 2)), ({}, dict(rs=0)),
    ({}, dict(rs=257)), ({}, dict(w=None)), ({}, dict(w=W + 8)), ({}, dict(out=None)), ({}, dict(out=OUT + 4)),
    ({}, dict(outs=OUTS)), ({}, dict(ro=None)), ({}, dict(ro=RO + 8)), ({}, dict(hs=255)), ({}, dict(rstd=RSTD + 2)),
    (dict(residual_dtype=NONE), dict(r=R)), (dict(residual_dtype=NONE), dict(ro=RO)), (dict(out_dtype=FP8), dict(outs=None)),
    (dict(out_dtype=FP8), dict(outs=OUTS + 1))])
def test_norm_arguments_refused(lib, cfg, args):
    log(lib)
    assert norm(lib, ncfg(**cfg), **args) == nat.AFD_E_ARG
    assert log(lib) == []


def test_norm_overlaps(lib):
    """100 rows of 256 bf16: 51200 bytes."""
    log(lib)
    c, size = ncfg(), 51200
    good = [dict(out=X), dict(ro=R), dict(ro=X), dict(out=X, ro=R), dict(out=X + size), dict(out=X - size),
            dict(ro=RO, out=RO + size), dict(ro=X, hs=264, xs=264)]
    for kw in good:
        assert norm(lib, c, **kw) == 0, kw
    bad = [dict(out=R), dict(out=X + 16), dict(out=X - 16), dict(out=RO), dict(ro=R + 16), dict(ro=X, out=X), dict(ro=W),
           dict(out=W), dict(rstd=X), dict(rstd=OUT + size - 4), dict(out=X, xs=264), dict(ro=R, rs=264), dict(ro=X, xs=264),
           dict(xs=512, out=X + 256 * 2)]
    for kw in bad:
        log(lib)
        assert norm(lib, c, **kw) == nat.AFD_E_ARG, kw
        assert log(lib) == []
    assert norm(lib, ncfg(x_dtype=FP32), out=X) == nat.AFD_E_ARG
    assert norm(lib, ncfg(residual_dtype=FP32), ro=X) == nat.AFD_E_ARG
    assert norm(lib, ncfg(out_dtype=FP8), out=X) == nat.AFD_E_ARG
    assert norm(lib, ncfg(out_dtype=FP8), outs=X) == nat.AFD_E_ARG
    assert norm(lib, ncfg(x_dtype=FP32, residual_dtype=FP32), ro=X) == 0
    assert norm(lib, ncfg(residual_dtype=NONE), out=X) == 0
    log(lib)


def test_norm_without_rows(lib):
    log(lib)
    assert norm(lib, ncfg(), 0, x=None, w=None, out=None) == 0
    assert grad(lib, ncfg(), 0, g=None, h=None, dw=None, ws=None, wsb=0) == 0
    assert log(lib) == []
    assert grad(lib, ncfg(), 0, g=None, h=None, rstd=None, w=None, dh=None, ws=None, wsb=0) == 0      # dweight is cleared
    assert "rows=0" in log(lib)[0]
    assert lib.afd_norm(None, 1, X, 8, None, 0, W, OUT, None, None, 0, None, None) == nat.AFD_E_ARG
    assert lib.afd_norm_grad_query(None, 1, ctypes.byref(ctypes.c_size_t())) == nat.AFD_E_ARG
    assert lib.afd_norm_grad_query(ctypes.byref(ncfg()), 1, None) == nat.AFD_E_ARG


@pytest.mark.parametrize("rows", [1, 100, 512, 513, 1024, 1025, 2049, ROWS])
@pytest.mark.parametrize("kw", [dict(), dict(hidden=16384), dict(hidden=8), dict(residual_dtype=FP32), dict(residual_dtype=NONE),
                                dict(residual_dtype=NONE, x_dtype=FP32)])
def test_norm_grad_workspace(lib, rows, kw):
    log(lib)
    c, need = ncfg(**kw), ctypes.c_size_t()
    assert lib.afd_norm_grad_query(ctypes.byref(c), rows, ctypes.byref(need)) == 0
    groups = 0 if rows <= (1024 if c.hidden <= 8192 else 512) else min(-(-rows // 4), 512)
    assert need.value == -(-groups * c.hidden * 4 // 256) * 256
    if groups:
        assert grad(lib, c, rows, wsb=need.value - 1) == nat.AFD_E_CAPACITY and log(lib) == []
    assert grad(lib, c, rows, ws=WS if groups else None, wsb=need.value) == 0
    h32 = c.residual_dtype == FP32 or c.residual_dtype == NONE and c.x_dtype == FP32
    assert f"norm_grad H={c.hidden} h32={int(h32)} w32=0 rows={rows}" in log(lib)[0]
    assert grad(lib, c, rows, dw=None, ws=None, wsb=0) == 0
    log(lib)


@pytest.mark.parametrize("args", [
    dict(rows=-1), dict(rows=1 << 24), dict(g=None), dict(g=X + 8), dict(gr=R + 4), dict(h=None), dict(h=OUT + 8),
    dict(hs=255), dict(hs=260), dict(w=None), dict(w=W + 2), dict(rstd=None), dict(rstd=RSTD + 2), dict(dh=None),
    dict(dh=RO + 8), dict(dw=DW + 2), dict(rows=1100, ws=None), dict(rows=1100, ws=WS + 16), dict(dh=OUT), dict(dh=X + 16), dict(dh=R - 16),
    dict(dw=RO), dict(dw=W), dict(rows=1100, ws=RO), dict(rows=1100, ws=X), dict(dh=RSTD)])
def test_norm_grad_arguments_refused(lib, args):
    log(lib)
    assert grad(lib, ncfg(), **args) == nat.AFD_E_ARG
    assert log(lib) == []


def test_norm_grad_in_place(lib):
    log(lib)
    assert grad(lib, ncfg(), dh=X) == 0 and grad(lib, ncfg(), dh=R) == 0 and grad(lib, ncfg(), gr=None) == 0
    assert grad(lib, ncfg(residual_dtype=FP32), dh=R) == 0
    assert grad(lib, ncfg(residual_dtype=FP32), dh=X) == nat.AFD_E_ARG      # float32 over bf16
    assert grad(lib, ncfg(out_dtype=FP8)) == nat.AFD_E_SHAPE
    assert len(log(lib)) == 4


# ------------------------------------------------------------------ routes --

L, IDS, WT, BIAS, LIVE, G, DL, LOSS, COUNTS, SLOPE = (i << 40 for i in range(20, 30))


def rcfg(**kw):
    c = dict(num_experts=96, topk=6, dtype=FP32, scoring=0, renormalize=1, scale=1.0)
    c.update(kw)
    return nat.RouteConfig(**c)


def route(lib, c, rows=100, **kw):
    a = dict(l=L, ls=c.num_experts, bias=None, live=None, ids=IDS, w=WT)
    a.update(kw)
    return lib.afd_route(ctypes.byref(c), rows, a["l"], a["ls"], a["bias"], a["live"], a["ids"], a["w"], None)


def route_grad(lib, c, rows=100, **kw):
    a = dict(g=G, l=L, ls=c.num_experts, ids=IDS, dl=DL)
    a.update(kw)
    return lib.afd_route_grad(ctypes.byref(c), rows, a["g"], a["l"], a["ls"], a["ids"], a["dl"], None)


def balance(lib, c, rows=100, **kw):
    a = dict(l=L, ls=c.num_experts, ids=IDS, co=1.0, loss=LOSS, counts=COUNTS, slope=SLOPE, ws=WS, wsb=1 << 40)
    a.update(kw)
    return lib.afd_balance(ctypes.byref(c), rows, a["l"], a["ls"], a["ids"], a["co"], a["loss"], a["counts"], a["slope"],
                           a["ws"], a["wsb"], None)


def balance_grad(lib, c, rows=100, **kw):
    a = dict(g=G, l=L, ls=c.num_experts, ids=IDS, slope=SLOPE, dl=DL)
    a.update(kw)
    return lib.afd_balance_grad(ctypes.byref(c), rows, a["g"], a["l"], a["ls"], a["ids"], a["slope"], a["dl"], None)


CALLS = [route, route_grad, balance, balance_grad]


@pytest.mark.parametrize("kw", [dict(), dict(num_experts=1, topk=1), dict(num_experts=512, topk=32), dict(dtype=BF16),
                                dict(scoring=1), dict(renormalize=0), dict(scale=-3e38), dict(scale=0.0)])
def test_routes_accepted(lib, kw):
    log(lib)
    c = rcfg(**kw)
    for call in CALLS:
        for rows in (1, ROWS):
            assert call(lib, c, rows) == 0
            line, = log(lib)
            assert line.startswith(f"{call.__name__} E={c.num_experts} K={c.topk} l32={int(c.dtype == FP32)} "
                                   f"sigmoid={c.scoring} ") and f"rows={rows} ls={c.num_experts}" in line
        assert call(lib, c, ls=2 ** 31 - 1) == 0
        log(lib)


@pytest.mark.parametrize("kw", [dict(num_experts=0), dict(num_experts=513), dict(topk=0), dict(topk=33), dict(topk=97),
                                dict(dtype=FP8), dict(dtype=3), dict(scoring=2), dict(scoring=-1), dict(renormalize=2),
                                dict(renormalize=-1), dict(scale=NAN), dict(scale=INF)])
def test_routes_shapes_refused(lib, kw):
    log(lib)
    need = ctypes.c_size_t()
    for call in CALLS:
        assert call(lib, rcfg(**kw)) == nat.AFD_E_SHAPE
    assert lib.afd_balance_query(ctypes.byref(rcfg(**kw)), 5, ctypes.byref(need)) == nat.AFD_E_SHAPE
    assert log(lib) == []


ROWS_BAD = [dict(rows=-1), dict(rows=1 << 24), dict(l=None), dict(l=L + 2), dict(ls=95), dict(ls=1 << 31), dict(ls=-96)]


@pytest.mark.parametrize("call,args", [(c, a) for c in CALLS for a in ROWS_BAD] + [
    (route, dict(ids=None)), (route, dict(ids=IDS + 1)), (route, dict(w=None)), (route, dict(w=WT + 2)),
    (route, dict(bias=BIAS + 2)), (route, dict(ids=WT)), (route, dict(ids=L)), (route, dict(w=L + 16)),
    (route, dict(bias=IDS)), (route, dict(live=WT + 4)),
    (route_grad, dict(g=None)), (route_grad, dict(g=G + 2)), (route_grad, dict(ids=None)), (route_grad, dict(dl=None)),
    (route_grad, dict(dl=DL + 2)), (route_grad, dict(dl=L)), (route_grad, dict(dl=G)), (route_grad, dict(dl=IDS - 4)),
    (balance, dict(ids=None)), (balance, dict(loss=None)), (balance, dict(loss=LOSS + 1)), (balance, dict(counts=None)),
    (balance, dict(slope=None)), (balance, dict(slope=COUNTS)), (balance, dict(loss=SLOPE + 4)), (balance, dict(counts=L)),
    (balance, dict(rows=1000, ws=None)), (balance, dict(rows=1000, ws=WS + 128)), (balance, dict(rows=1000, ws=IDS)),
    (balance, dict(rows=1000, ws=SLOPE)),
    (balance, dict(co=NAN)), (balance, dict(co=INF)),
    (balance_grad, dict(g=None)), (balance_grad, dict(slope=None)), (balance_grad, dict(slope=SLOPE + 2)),
    (balance_grad, dict(ids=IDS + 2)), (balance_grad, dict(dl=None)), (balance_grad, dict(dl=L)), (balance_grad, dict(dl=SLOPE)),
    (balance_grad, dict(dl=G)), (balance_grad, dict(dl=IDS))])
def test_routes_arguments_refused(lib, call, args):
    log(lib)
    assert call(lib, rcfg(), **args) == nat.AFD_E_ARG
    assert log(lib) == []


def test_bf16_logits_need_two_bytes(lib):
    log(lib)
    c = rcfg(dtype=BF16)
    for call in CALLS:
        assert call(lib, c, l=L + 2) == 0 and call(lib, c, l=L + 1) == nat.AFD_E_ARG
    assert route_grad(lib, c, dl=DL + 2) == 0
    log(lib)


def test_routes_without_rows(lib):
    log(lib)
    c = rcfg()
    assert route(lib, c, 0, l=None, ids=None, w=None) == 0
    assert route_grad(lib, c, 0, g=None, l=None, ids=None, dl=None) == 0
    assert balance_grad(lib, c, 0, g=None, l=None, ids=None, slope=None, dl=None) == 0
    assert log(lib) == []
    assert balance(lib, c, 0, l=None, ids=None, ws=None, wsb=0) == 0       # loss, counts and slope are cleared
    assert "groups=0" in log(lib)[0]


@pytest.mark.parametrize("E,each", [(1, 16), (96, 16), (128, 16), (129, 8), (256, 8), (257, 4), (512, 4)])
@pytest.mark.parametrize("rows", [1, 96, 97, 192, 193, 384, 385, 513, 4096, 8192, 8193, ROWS])
def test_balance_workspace(lib, E, each, rows):
    """The first launch's sums, counts and totals, the loss's parts and the count of the done."""
    log(lib)
    c, need = rcfg(num_experts=E, topk=1), ctypes.c_size_t()
    assert lib.afd_balance_query(ctypes.byref(c), rows, ctypes.byref(need)) == 0
    if rows <= 24 * each:                            # one workgroup's
        assert need.value == 0
        assert balance(lib, c, rows, ws=None, wsb=0) == 0
        assert " groups=1 " in log(lib)[0]
        return
    groups = min(-(-rows // each), 256)
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    sizes = [up(groups * E * 4), up(groups * E * 4), up(groups * 8), up(-(-E // 16) * 8), 256]
    assert need.value == sum(sizes)
    assert balance(lib, c, rows, wsb=need.value - 1) == nat.AFD_E_CAPACITY and log(lib) == []
    assert balance(lib, c, rows, wsb=need.value) == 0
    line, = log(lib)
    assert f"groups={groups} wide={int(rows > 512 * each)}" in line
    at = [int(line.split(f" {k}=")[1].split()[0], 16) for k in ("share", "count", "totals", "part", "done")]
    assert at == [WS + sum(sizes[:i]) for i in range(5)]


def test_launch_failures_are_reported(lib):
    lib.afd_fake_set_fail(1)
    try:
        assert norm(lib, ncfg()) == nat.AFD_E_HIP and grad(lib, ncfg()) == nat.AFD_E_HIP
        assert [call(lib, rcfg()) for call in CALLS] == [nat.AFD_E_HIP] * 4
    finally:
        lib.afd_fake_set_fail(0)
        log(lib)
