"""The rows per expert by which the experts' kernels are chosen (over the
recording backend): the caller's number where there is one, and what
worker_experts passes."""
import ctypes
import re

import pytest
import torch

import combine_layout_amd as afd
from combine_layout_amd import _native as nat
from combine_layout_amd import buffer as buffer_module
from tests.test_experts_host import LOW, call, fcfg, ffn, log, pcfg


@pytest.fixture(scope="module")
def lib():
    return nat.load_fake()


def chosen(lib):
    return [tuple(map(int, re.search(r" each=(\d+) live=(\d+) ", line).groups())) for line in log(lib)]


@pytest.mark.parametrize("E,alpha,rows,hint,each,live", [
    # rows that the host counted, all of them padding or all of them live: the bound cannot tell
    (64, 128, 64 * 128, 0, 0, 8192), (64, 128, 64 * 128, 100, 100, 6400), (64, 128, 64 * 128, 1, 1, 64),
    # an arena's bound: half of its choices, or what one partition of many gets
    (64, 64, 2048 + 64 * 63, 0, 16, 6080), (16, 64, 2048 + 16 * 63, 0, 64, 3056), (16, 64, 2048 + 16 * 63, 16, 16, 256),
    # one token; no more rows than there are
    (96, 64, 8 + 96 * 63, 1, 1, 96), (96, 64, 8 + 96 * 63, 0, 0, 6056), (4, 1, 10, 2 ** 31 - 1, 3, 10), (4, 1, 10, 0, 1, 10),
    (512, 2 ** 31 - 1, (1 << 24) - 1, 0, 0, (1 << 24) - 1)])
def test_expected_rows(lib, E, alpha, rows, hint, each, live):
    log(lib)
    for kw in (dict(), LOW):
        assert call(lib, pcfg(num_experts=E, alignment=alpha, k=64, n=16, rows_per_expert=hint, **kw), rows=rows, x=1 << 40,
                    out=1 << 41, wsb=1 << 40) == 0
        assert ffn(lib, fcfg(num_experts=E, alignment=alpha, rows_per_expert=hint, **kw), rows=rows, wsb=1 << 40) == 0
    assert chosen(lib) == [(each, live)] * 6


def test_negative_refused(lib):
    log(lib)
    need = ctypes.c_size_t()
    for c, query in ((pcfg(rows_per_expert=-1), lib.afd_product_query), (fcfg(rows_per_expert=-1), lib.afd_ffn_query)):
        assert query(ctypes.byref(c), 5, ctypes.byref(need)) == nat.AFD_E_SHAPE
    assert call(lib, pcfg(rows_per_expert=-1)) == nat.AFD_E_SHAPE and ffn(lib, fcfg(rows_per_expert=-1)) == nat.AFD_E_SHAPE
    assert log(lib) == []


@pytest.mark.parametrize("T,want", [((128, 128), 16), ((1, 0), 1), ((0, 0), 0), ((2048, 2047), 256)])
def test_worker_experts_expects_evenly_spread_choices(lib, monkeypatch, T, want):
    buf = afd.Buffer.__new__(afd.Buffer)
    buf.ctx, buf.alpha, buf._T, buf.K, buf.E = None, 64, list(T), 8, 128

    class Lib:
        @staticmethod
        def afd_get_round_info(ctx, info):
            info._obj.round = 7
            return 0

    buf.lib = Lib
    seen = {}
    monkeypatch.setattr(buffer_module._experts, "expert_ffn", lambda *a, **kw: seen.update(kw))
    rec = afd.Received(torch.zeros(1, 1), None, None, None, nat.Receipt(7, 0, 0), 1, None)
    buf.worker_experts(0, rec, None)
    assert seen["rows_per_expert"] == want and seen["alignment"] == 64


@pytest.mark.parametrize("at,what", [(0, "num_experts"), (1, "alignment"), (2, "k"), (3, "n"), (7, "num_adapters"), (8, "rank"),
                                     (10, "rows_per_expert")])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 64, -1])
def test_what_no_int32_holds_is_refused(monkeypatch, lib, at, what, value):
    """A width of 2^32 + 64 is not one of 64."""
    from combine_layout_amd import experts
    monkeypatch.setattr(nat, "load", nat.load_fake)
    good = [4, 16, 64, 64, nat.AFD_BF16, nat.AFD_BF16, 0, 2, 8, 0, 0]
    assert experts._product_plan(10, *good)[0].k == 64
    good[at] = value
    with pytest.raises(ValueError, match=what):
        experts._product_plan(10, *good)
    network = [4, 16, 64, 64, nat.AFD_BF16, 2, 8, 0, 0]
    assert experts._ffn_plan(10, *network)[0].inner == 64
    fields = [name for name, _ in nat.FfnConfig._fields_]
    name = {"k": "hidden", "n": "inner"}.get(what, what)
    network[fields.index(name)] = value
    with pytest.raises(ValueError, match=name):
        experts._ffn_plan(10, *network)
