"""Workspace sizes and launches of the experts' calls at the largest accepted
rows, widths, ranks and numbers (over the recording backend): every size is the
exact one, in 64 bits."""
import ctypes

import pytest

from combine_layout_amd import _native as nat
from tests.test_experts_host import LOW, call, fcfg, ffn, log, pcfg, weights

ROWS = (1 << 24) - 1
TOP = dict(num_adapters=65536, rank=128)


@pytest.fixture(scope="module")
def lib():
    return nat.load_fake()


def align(v):
    return -(-v // 256) * 256


def need(query, c, rows):
    n = ctypes.c_size_t()
    assert query(ctypes.byref(c), rows, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("kw,kinds", [(dict(k=1 << 21, n=16 * 31), 1), (dict(k=64, n=(1 << 23) - 16, activation=1), 2),
                                      (dict(k=1 << 21, n=16 * 63, dtype=1), 1),
                                      (dict(k=128, n=(1 << 23) - 128, dtype=1, out_dtype=1, activation=1), 2)])
@pytest.mark.parametrize("rows", [1, 255, ROWS])
def test_product(lib, kw, kinds, rows):
    log(lib)
    assert need(lib.afd_product_query, pcfg(num_experts=512, alignment=2 ** 31 - 1, **kw), rows) == 0
    c = pcfg(num_experts=512, alignment=2 ** 31 - 1, **TOP, **kw)
    size = need(lib.afd_product_query, c, rows)
    assert size == align(rows * 128 * kinds * 4)
    # x of up to 2^46 bytes lies in front of out
    fake = dict(rows=rows, x=1 << 47, out=1 << 48, wsb=size)
    assert call(lib, c, **fake) == 0
    assert call(lib, c, **dict(fake, wsb=size - 1)) == nat.AFD_E_CAPACITY
    assert call(lib, c, **dict(fake, rows=ROWS + 1)) == nat.AFD_E_ARG
    line, = log(lib)
    assert f"rows={rows}" in line and f"k={c.k} n={c.n}" in line
    # the first width whose expert holds 2^31 bytes
    step, row = 128 if c.out_dtype else 16, kinds * c.k * (1 if c.dtype else 2)
    over = -(-(1 << 31) // row // step) * step
    assert call(lib, pcfg(num_experts=512, **dict(kw, n=over)), **fake) == nat.AFD_E_SHAPE
    assert call(lib, pcfg(num_experts=512, **dict(kw, n=over - step)), **fake) == 0
    log(lib)


@pytest.mark.parametrize("kw", [dict(hidden=192, inner=1 << 21), dict(hidden=1 << 21, inner=192),
                                dict(hidden=384, inner=1 << 21, dtype=1), dict(hidden=1 << 21, inner=384, dtype=1)])
@pytest.mark.parametrize("rows", [1, 255, ROWS])
@pytest.mark.parametrize("low", [dict(), TOP, dict(LOW, rank=8)])
def test_network(lib, kw, rows, low):
    log(lib)
    c = fcfg(num_experts=512, alignment=2 ** 31 - 1, **low, **kw)
    fp8 = c.dtype == 1
    size = need(lib.afd_ffn_query, c, rows)
    assert size == align(rows * c.inner * (1 if fp8 else 2)) + (align(rows * (c.inner // 128) * 4) if fp8 else 0) + \
        align(rows * c.rank * 2 * 4)
    assert ffn(lib, c, rows=rows, wsb=size - 1) == nat.AFD_E_CAPACITY
    assert ffn(lib, c, rows=rows, wsb=size) == 0
    assert len(log(lib)) == 2


@pytest.mark.parametrize("kw,row_bytes", [(dict(k=64, n=(1 << 24) - 16), 128), (dict(k=1 << 21, n=496), 1 << 22),
                                          (dict(k=128, n=(1 << 24) - 16, dtype=1), 128)])
def test_packing(lib, kw, row_bytes):
    log(lib)
    c = pcfg(num_experts=512, **kw)
    w, out = 9 << 20, 1 << 50
    assert lib.afd_pack_weights(ctypes.byref(c), w, out, None) == 0
    assert log(lib) == [f"pack {hex(w)}->{hex(out)} rows={512 * c.n} row_bytes={row_bytes}"]


def test_overlap_at_the_end_of_the_address_space(lib):
    """The extents are compared in addresses, not in pointers that might wrap."""
    log(lib)
    c = pcfg(k=64, n=16)
    top = (1 << 64) - 4096
    assert call(lib, c, rows=16, x=top, out=top + 2048) == 0      # x [16, 64] holds 2048 bytes
    assert call(lib, c, rows=16, x=top, out=top + 2032) == nat.AFD_E_ARG
    assert weights().w and len(log(lib)) == 1
