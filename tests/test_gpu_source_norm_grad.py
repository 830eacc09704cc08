"""The norm's gradient of many rows: with and without the residual's gradient and
dweight, past the rows that its grid holds at once, and the same dh either way."""
import pytest
import torch

from tests import source_ref as ref
from tests.test_gpu_source import BF, F32, _afd, _gapped, _gen, _print, _rand

pytestmark = pytest.mark.gpu


def _inputs(T, H, ht):
    g = _gen(T + H)
    h, w, dy, dr = _rand(g, T, H, dtype=ht), 1 + _rand(g, H, std=0.3), _rand(g, T, H, dtype=BF), _rand(g, T, H, dtype=ht)
    return h, w, dy, dr, (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()


@pytest.mark.parametrize("T,H", [(1024, 2048), (1025, 2048), (4097, 2048), (1025, 1032), (2049, 1504), (4100, 512), (1030, 1024),
                                 (1100, 4096), (1025, 8192), (513, 16384)])
@pytest.mark.parametrize("ht", [BF, F32])
@pytest.mark.parametrize("res", [False, True])
def test_dh_is_the_same_with_and_without_dweight(T, H, ht, res):
    afd = _afd()
    _print("dh", T, H, ht, res)
    h, w, dy, dr, rstd = (t.cuda() for t in _inputs(T, H, ht))
    kw = dict(grad_residual=dr) if res else {}
    dh, dw = afd.rms_norm_grad(dy, h, w, rstd, **kw)
    alone, none = afd.rms_norm_grad(dy, h, w, rstd, weight_grad=False, **kw)
    assert dw is not None and none is None
    assert torch.equal(dh, alone)


@pytest.mark.parametrize("T,H", [(4099, 2048), (9000, 72), (5001, 1024), (2600, 4104), (2100, 8192)])
@pytest.mark.parametrize("ht", [BF, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("weight_grad", [False, True])
def test_many_rows(T, H, ht, res, weight_grad):
    afd = _afd()
    _print("rows", T, H, ht, res, weight_grad)
    h, w, dy, dr, rstd = _inputs(T, H, ht)
    dh, dw = afd.rms_norm_grad(dy.cuda(), _gapped(h, 8), w.cuda(), rstd.cuda(), weight_grad=weight_grad,
                               grad_residual=dr.cuda() if res else None)
    want, tol, wantw, tolw = ref.norm_grad(dy.double(), h.double(), w.double(), rstd.double(), dr.double() if res else None)
    ref.check(dh, want, ref.rounded(want, tol, ht), "dh")
    if weight_grad:
        ref.check(dw, wantw, tolw + ref.U * wantw.abs(), "dweight")
    else:
        assert dw is None
