"""What the Python calls of the source's side refuse before they reach the GPU
(on host and meta tensors, which are refused as well)."""
import pytest
import torch
from torch.autograd import forward_ad

import combine_layout_amd as afd

BF = torch.bfloat16
X, W, L = torch.zeros(4, 256, dtype=BF), torch.ones(256, dtype=BF), torch.zeros(4, 8)
IDS, ONE = torch.zeros(4, 2, dtype=torch.int32), torch.ones(())

HOST = {
    "rms_norm": lambda f: afd.rms_norm(f(X), W),
    "rms_norm weight": lambda f: afd.rms_norm(X, f(W)),
    "rms_norm residual": lambda f: afd.rms_norm(X, W, f(X)),
    "rms_norm_grad": lambda f: afd.rms_norm_grad(f(X), X, W, torch.ones(4)),
    "rms_norm_grad h": lambda f: afd.rms_norm_grad(X, f(X), W, torch.ones(4)),
    "route_tokens": lambda f: afd.route_tokens(f(L), 2),
    "route_tokens_grad": lambda f: afd.route_tokens_grad(torch.ones(4, 2), f(L), IDS),
    "balance_loss": lambda f: afd.balance_loss(f(L), IDS),
    "balance_loss_grad": lambda f: afd.balance_loss_grad(ONE, f(L), IDS, torch.ones(8)),
}


@pytest.mark.parametrize("name", list(HOST))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="GPU|cpu"):
        HOST[name](lambda t: t)


@pytest.mark.parametrize("name", list(HOST))
def test_dual_tensors_are_refused(name):
    with forward_ad.dual_level():
        for grad in (False, True):
            with torch.set_grad_enabled(grad):
                with pytest.raises(ValueError, match="forward gradients"):
                    HOST[name](lambda t: forward_ad.make_dual(t, torch.ones_like(t)))


@pytest.mark.parametrize("call", [
    lambda t: afd.rms_norm(X, W, out=t(X)), lambda t: afd.rms_norm(X, W, out_scales=t(L)),
    lambda t: afd.rms_norm(X, W, X, residual_out=t(X)), lambda t: afd.rms_norm_grad(t(X), X, W, torch.ones(4)),
    lambda t: afd.rms_norm_grad(X, t(X), W, torch.ones(4)), lambda t: afd.rms_norm_grad(X, X, t(W), torch.ones(4)),
    lambda t: afd.rms_norm_grad(X, X, W, t(torch.ones(4))), lambda t: afd.rms_norm_grad(X, X, W, ONE, grad_residual=t(X)),
    lambda t: afd.rms_norm_grad(X, X, W, ONE, out=t(X)), lambda t: afd.route_tokens(L, 2, bias=t(torch.ones(8))),
    lambda t: afd.route_tokens(L, 2, weights=t(torch.ones(4, 2))), lambda t: afd.route_tokens_grad(t(L), L, IDS),
    lambda t: afd.route_tokens_grad(L, t(L), IDS), lambda t: afd.balance_loss_grad(t(ONE), L, IDS, torch.ones(8)),
    lambda t: afd.balance_loss_grad(ONE, t(L), IDS, torch.ones(8)), lambda t: afd.balance_loss_grad(ONE, L, IDS, t(ONE))])
def test_arguments_that_have_no_gradient(call):
    asks = lambda t: t.clone().requires_grad_()  # noqa: E731
    with pytest.raises(ValueError, match="no gradient reaches"):
        call(asks)
    with torch.no_grad(), pytest.raises(ValueError) as e:
        call(asks)
    assert "gradient" not in str(e.value)


def test_given_outputs_are_not_recorded():
    x, l = X.clone().requires_grad_(), L.clone().requires_grad_()
    for kw in (dict(out=X), dict(dtype=torch.float8_e4m3fn), dict(residual_out=X)):
        with pytest.raises(ValueError, match="have no gradient"):
            afd.rms_norm(x, W, X, **kw)
    for kw in (dict(ids=IDS), dict(weights=torch.ones(4, 2))):
        with pytest.raises(ValueError, match="have no gradient"):
            afd.route_tokens(l, 2, **kw)


def test_names():
    """The public names, and the library's signatures behind them."""
    from combine_layout_amd import _native as nat
    for name in ("rms_norm", "rms_norm_grad", "route_tokens", "route_tokens_grad", "balance_loss", "balance_loss_grad",
                 "Normed", "Routes", "Balance"):
        assert hasattr(afd, name)
    assert {"source_norm", "source_route"} <= set(dir(afd.Buffer))
    assert {"afd_norm", "afd_norm_grad", "afd_route", "afd_route_grad", "afd_balance", "afd_balance_grad"} <= set(nat.SIGNATURES)
