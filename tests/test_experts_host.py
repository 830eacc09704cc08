"""Host checks of the experts' entry points (over the recording backend): the
refusals, the workspace sizes and the launches they lead to.  Refused calls
launch nothing."""
import ctypes

import pytest

from combine_layout_amd import _native as nat
from tests.test_host_core import FAKE_WS, Ctx  # noqa: F401


@pytest.fixture(scope="module")
def lib():
    return nat.load_fake()


def log(lib):
    out = []
    for i in range(lib.afd_fake_log_size()):
        b = ctypes.create_string_buffer(1024)
        lib.afd_fake_log_get(i, b, 1024)
        out.append(b.value.decode())
    lib.afd_fake_log_clear()
    return out


def pcfg(**kw):
    c = dict(num_experts=4, alignment=16, k=256, n=128, dtype=0, out_dtype=0, activation=0, num_adapters=0, rank=0, weight_layout=0)
    c.update(kw)
    return nat.ProductConfig(**c)


X, XS, ENDS, TAGS, OUT, OUTS, WS = (i << 20 for i in range(1, 8))


def weights(fp8=False, low=False, **kw):
    w = nat.ProductWeights(w=9 << 20, w_scales=(10 << 20) if fp8 else None, a=(11 << 20) if low else None,
                           b=(12 << 20) if low else None, scaling=(13 << 20) if low else None)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def call(lib, c, rows=100, x=X, xs="auto", ends=ENDS, tags="auto", w="auto", out=OUT, outs="auto", ws=WS, wsb=1 << 30):
    fp8, low = c.dtype == 1, c.num_adapters > 0
    xs = (XS if fp8 else None) if xs == "auto" else xs
    tags = (TAGS if low else None) if tags == "auto" else tags
    outs = (OUTS if c.out_dtype == 1 else None) if outs == "auto" else outs
    w = weights(fp8, low) if w == "auto" else w
    return lib.afd_expert_product(ctypes.byref(c), rows, x, xs, ends, tags, ctypes.byref(w) if w is not None else None, out,
                                  outs, ws, wsb, None)


FP8G = dict(dtype=1, activation=1, n=128)
LOW = dict(num_adapters=3, rank=16)


@pytest.mark.parametrize("kw", [dict(), dict(k=64, n=16), dict(activation=1, n=48), dict(dtype=1, n=16), FP8G,
                                dict(FP8G, out_dtype=1), LOW, dict(FP8G, out_dtype=1, **LOW),
                                dict(num_adapters=65536, rank=128), dict(num_experts=512), dict(alignment=2 ** 31 - 1),
                                dict(weight_layout=1)])
def test_accepted(lib, kw):
    log(lib)
    c = pcfg(**kw)
    assert call(lib, c) == 0
    lines = log(lib)
    assert len(lines) == 1 and lines[0].startswith(f"product E={c.num_experts} alpha={c.alignment} k={c.k} n={c.n} ")
    assert f"nad={c.num_adapters} rank={c.rank} packed={c.weight_layout} rows=100" in lines[0]


@pytest.mark.parametrize("kw", [
    dict(num_experts=0), dict(num_experts=513), dict(alignment=0), dict(k=0), dict(k=32), dict(k=-64), dict(dtype=1, k=64),
    dict(k=(1 << 21) + 64, n=16), dict(n=0), dict(n=8), dict(n=24), dict(dtype=2), dict(dtype=-1), dict(activation=2), dict(out_dtype=1),
    dict(dtype=1, out_dtype=1), dict(FP8G, out_dtype=2), dict(activation=1, out_dtype=1), dict(FP8G, n=64),
    dict(num_adapters=-1), dict(num_adapters=3), dict(rank=16), dict(LOW, rank=4), dict(LOW, rank=20), dict(LOW, rank=136),
    dict(num_adapters=65537, rank=16), dict(k=1 << 20, n=1 << 10), dict(k=1 << 19, n=1 << 10, activation=1),
    dict(n=2 ** 31 - 16), dict(weight_layout=2), dict(weight_layout=-1)])
def test_shapes_refused(lib, kw):
    log(lib)
    c = pcfg(**kw)
    need = ctypes.c_size_t()
    assert call(lib, c) == nat.AFD_E_SHAPE
    assert lib.afd_product_query(ctypes.byref(c), 5, ctypes.byref(need)) == nat.AFD_E_SHAPE
    assert log(lib) == []


@pytest.mark.parametrize("kw,args", [
    ({}, dict(rows=-1)), ({}, dict(rows=1 << 24)), ({}, dict(x=None)), ({}, dict(x=X + 8)), ({}, dict(ends=None)),
    ({}, dict(ends=ENDS + 2)), ({}, dict(out=None)), ({}, dict(out=OUT + 2)), ({}, dict(w=None)), ({}, dict(xs=XS)),
    ({}, dict(outs=OUTS)), ({}, dict(tags=TAGS)), ({}, dict(w=weights(w=None))), ({}, dict(w=weights(w=(9 << 20) + 4))),
    ({}, dict(w=weights(fp8=True))), ({}, dict(w=weights(low=True))), (FP8G, dict(xs=None)), (FP8G, dict(xs=XS + 1)),
    (FP8G, dict(w=weights())), (dict(FP8G, out_dtype=1), dict(outs=None)), (LOW, dict(tags=None)),
    (LOW, dict(w=weights(low=True, a=None))), (LOW, dict(w=weights(low=True, b=(12 << 20) + 2))),
    (LOW, dict(w=weights(low=True, scaling=None))), (LOW, dict(w=weights())), (LOW, dict(ws=None)),
    (LOW, dict(ws=WS + 16))])
def test_arguments_refused(lib, kw, args):
    log(lib)
    assert call(lib, pcfg(**kw), **args) == nat.AFD_E_ARG
    assert log(lib) == []


def test_null_and_no_rows(lib):
    log(lib)
    need = ctypes.c_size_t()
    w = weights()
    assert lib.afd_expert_product(None, 1, X, None, ENDS, None, ctypes.byref(w), OUT, None, None, 0, None) == nat.AFD_E_ARG
    assert lib.afd_product_query(None, 1, ctypes.byref(need)) == nat.AFD_E_ARG
    c = pcfg()
    assert lib.afd_product_query(ctypes.byref(c), 1, None) == nat.AFD_E_ARG
    assert call(lib, c, rows=0, x=None, ends=None, out=None, w=None) == 0
    assert log(lib) == []


def test_workspace(lib):
    log(lib)
    need = ctypes.c_size_t()
    c = pcfg()
    assert lib.afd_product_query(ctypes.byref(c), 1000, ctypes.byref(need)) == 0 and need.value == 0
    assert call(lib, c, ws=None, wsb=0) == 0
    for kw, per in ((LOW, 16 * 4), (dict(LOW, activation=1), 2 * 16 * 4)):
        c = pcfg(**kw)
        assert lib.afd_product_query(ctypes.byref(c), 1000, ctypes.byref(need)) == 0
        assert need.value >= 1000 * per and need.value % 256 == 0
        log(lib)
        assert call(lib, c, rows=1000, wsb=need.value - 1) == nat.AFD_E_CAPACITY
        assert log(lib) == []
        assert call(lib, c, rows=1000, wsb=need.value) == 0


def test_pack(lib):
    log(lib)
    c = pcfg(activation=1, n=48, k=320)
    w, out = 9 << 20, 30 << 20
    assert lib.afd_pack_weights(ctypes.byref(c), w, out, None) == 0
    assert log(lib) == [f"pack {hex(w)}->{hex(out)} rows={4 * 96} row_bytes=640"]
    for a, b in ((None, out), (w, None), (w, w), (w + 8, out), (w, out + 4)):
        assert lib.afd_pack_weights(ctypes.byref(c), a, b, None) == nat.AFD_E_ARG
    assert lib.afd_pack_weights(ctypes.byref(pcfg(k=100)), w, out, None) == nat.AFD_E_SHAPE
    assert lib.afd_pack_weights(None, w, out, None) == nat.AFD_E_ARG
    assert log(lib) == []


def fcfg(**kw):
    c = dict(num_experts=4, alignment=16, hidden=256, inner=128, dtype=0, num_adapters=0, rank=0)
    c.update(kw)
    return nat.FfnConfig(**c)


def ffn(lib, c, rows=100, wsb=1 << 30, up=None, down=None, ws=WS, **kw):
    fp8, low = c.dtype == 1, c.num_adapters > 0
    up, down = up or weights(fp8, low), down or weights(fp8, low)
    a = dict(x=X, xs=XS if fp8 else None, ends=ENDS, tags=TAGS if low else None, out=OUT)
    a.update(kw)
    return lib.afd_expert_ffn(ctypes.byref(c), rows, a["x"], a["xs"], a["ends"], a["tags"], ctypes.byref(up),
                              ctypes.byref(down), a["out"], ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(), dict(dtype=1), LOW, dict(LOW, dtype=1)])
def test_ffn_launches(lib, kw):
    log(lib)
    c = fcfg(**kw)
    need = ctypes.c_size_t()
    assert lib.afd_ffn_query(ctypes.byref(c), 100, ctypes.byref(need)) == 0
    assert ffn(lib, c, wsb=need.value - 1) == nat.AFD_E_CAPACITY and log(lib) == []
    assert ffn(lib, c, wsb=need.value) == 0
    up, down = log(lib)
    f8 = c.dtype
    assert f"k=256 n=128 fp8={f8} out8={f8} gated=1" in up and f"out={hex(WS)}" in up and f"x={hex(X)}" in up
    assert f"k=128 n=256 fp8={f8} out8=0 gated=0" in down and f"x={hex(WS)}" in down and f"out={hex(OUT)}" in down
    h = 100 * 128 * (1 if f8 else 2)
    if f8:      # the hidden rows' scales lie behind them, the adapters' rows behind those
        outs = int(up.split("outs=")[1].split()[0], 16)
        assert outs >= WS + h and outs + 100 * 4 <= WS + need.value
        h = outs + 400 - WS
    if c.num_adapters:
        t = int(up.split(" t=")[1], 16)
        assert t >= WS + h and t + 100 * 2 * 16 * 4 <= WS + need.value and t % 256 == 0
    log(lib)


@pytest.mark.parametrize("kw", [dict(hidden=32), dict(inner=0), dict(inner=32), dict(dtype=1, inner=64), dict(dtype=1, hidden=192),
                                dict(num_experts=0), dict(rank=8)])
def test_ffn_shapes_refused(lib, kw):
    log(lib)
    need = ctypes.c_size_t()
    assert lib.afd_ffn_query(ctypes.byref(fcfg(**kw)), 100, ctypes.byref(need)) == nat.AFD_E_SHAPE
    assert ffn(lib, fcfg(**kw)) == nat.AFD_E_SHAPE
    assert log(lib) == []


def test_ffn_arguments_refused(lib):
    log(lib)
    for kw in (dict(x=None), dict(x=X + 4), dict(ends=None), dict(out=None), dict(xs=XS), dict(tags=TAGS), dict(ws=None),
               dict(ws=WS + 64), dict(up=weights(w=None)), dict(down=weights(fp8=True)), dict(rows=-5)):
        assert ffn(lib, fcfg(), **kw) == nat.AFD_E_ARG, kw
    assert ffn(lib, fcfg(), rows=0, ws=None, x=None) == 0
    assert log(lib) == []


def test_launch_failure_is_reported(lib):
    lib.afd_fake_set_fail(1)
    try:
        assert call(lib, pcfg()) == nat.AFD_E_HIP
        assert ffn(lib, fcfg()) == nat.AFD_E_HIP
    finally:
        lib.afd_fake_set_fail(0)
        log(lib)


def test_worker_tags_order_and_arguments(lib):
    c = nat.Config(2, 2, 8, 2, 256, 4, 16, 0, 0, 0)
    x = Ctx(lib, c)
    tags = (ctypes.c_void_p * 2)(0x100, 0x200)
    out = 0xA000000

    def tag(f, rec, rows=None, t=tags, o=out, partition=None, rnd=None):
        r = nat.Receipt(rec.receipt.round if rnd is None else rnd, rec.receipt.partition if partition is None else partition, 0)
        return lib.afd_worker_tags(x.ctx, f, t, o, rec.receive_rows if rows is None else rows, ctypes.byref(r), None)

    assert x.dispatch(0, 4) == 0 and x.dispatch(1, 0) == 0
    none = nat.Receive()
    assert tag(0, none) == nat.AFD_E_ORDER                  # nothing received yet
    st, rec, _ = x.receive(0)
    assert st == 0
    log(lib)
    assert tag(0, rec) == 0
    assert log(lib) == [f"tags f=0 ntok=4 out={hex(out)}"]
    assert tag(1, rec) == nat.AFD_E_ORDER                   # not received
    assert tag(0, rec, partition=1) == nat.AFD_E_ORDER
    assert tag(0, rec, rnd=99) == nat.AFD_E_ORDER
    assert tag(2, rec) == nat.AFD_E_ARG and tag(-1, rec) == nat.AFD_E_ARG
    assert tag(0, rec, rows=rec.receive_rows - 1) == nat.AFD_E_SHAPE
    assert tag(0, rec, o=None) == nat.AFD_E_ARG and tag(0, rec, o=out + 2) == nat.AFD_E_ARG
    assert tag(0, rec, t=(ctypes.c_void_p * 2)(None, 0x200)) == nat.AFD_E_ARG
    assert tag(0, rec, t=(ctypes.c_void_p * 2)(0x101, None)) == nat.AFD_E_ARG
    assert tag(0, rec, t=(ctypes.c_void_p * 2)(0x100, None)) == 0     # source 1 is empty
    assert tag(0, rec, t=None) == nat.AFD_E_ARG
    assert x.reply(0, rec) == 0
    assert tag(0, rec) == nat.AFD_E_ORDER                   # replied
    st, rec1, _ = x.receive(1)
    assert st == 0 and tag(1, rec1) == 0                    # the other partition still may
    assert x.reply(1, rec1) == 0
    assert tag(1, rec1) == nat.AFD_E_ORDER
    x.destroy()
    log(lib)


def test_python_calls_refuse_host_tensors():
    import torch

    import combine_layout_amd as afd
    x, ends, w = torch.zeros((4, 64)).bfloat16(), torch.tensor([4], dtype=torch.int32), torch.zeros((1, 16, 64)).bfloat16()
    with pytest.raises(ValueError):
        afd.expert_product(x, ends, w)
    with pytest.raises(ValueError):
        afd.expert_ffn(x, ends, None)
    with pytest.raises(ValueError):
        afd.pack_weights(w)


def test_out_over_x_refused(lib):
    """x [100, 256] bf16 holds 51200 bytes, out [100, 128] 25600."""
    log(lib)
    for out in (X, X + 51200 - 16, X - 25600 + 16):
        assert call(lib, pcfg(), out=out) == nat.AFD_E_ARG
    assert not log(lib)
    for out in (X + 51200, X - 25600):
        assert call(lib, pcfg(), out=out) == 0
    assert len(log(lib)) == 2
