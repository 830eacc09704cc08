"""What the Python calls of the source's side tell autograd of the memory they are
given: every output's version counter rises, no input's does (the library's launch
is left out, so that it runs on any host)."""
import contextlib

import pytest
import torch

import combine_layout_amd as afd
from combine_layout_amd import source

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def no_launch(monkeypatch):
    class Library:
        def __getattr__(self, name):
            return name
    monkeypatch.setattr(source.nat, "load", lambda: Library())
    monkeypatch.setattr(source, "_launch", lambda *a: 0)
    for plans, plan, made in (("_norms", "_norm_plan", (None, 256, 256, 256)), ("_norm_grads", "_norm_grad_plan", (None, 256, 0)),
                              ("_routes", "_route_plan", (source.nat.RouteConfig(topk=2), 8)),
                              ("_routes", "_route_grad_plan", (None, 8)), ("_balances", "_balance_plan", (None, 8, 0)),
                              ("_balances", "_balance_grad_plan", (None, 8))):
        monkeypatch.setattr(source, plans, {})
        monkeypatch.setattr(source, plan, lambda *a, made=made: made)


def _t():
    return dict(x=torch.zeros(4, 256, dtype=BF), w=torch.ones(256), r=torch.zeros(4, 256, dtype=BF), l=torch.zeros(4, 8),
                ids=torch.zeros(4, 2, dtype=torch.int32), wt=torch.zeros(4, 2), rstd=torch.ones(4), bias=torch.zeros(8),
                live=torch.ones(4, dtype=torch.bool), g=torch.ones(()), slope=torch.ones(8), q=torch.zeros(4, 256).to(F8),
                s=torch.zeros(4, 2), out=torch.zeros(4, 256, dtype=BF), dl=torch.zeros(4, 8))


# the call, and the tensors that it is given to write
CALLS = {
    "norm out": (lambda t: afd.rms_norm(t["x"], t["w"], out=t["out"]), "out"),
    "norm over x": (lambda t: afd.rms_norm(t["x"], t["w"], out=t["x"]), "x"),
    "norm residual_out": (lambda t: afd.rms_norm(t["x"], t["w"], t["r"], residual_out=t["out"]), "out"),
    "norm over the residual": (lambda t: afd.rms_norm(t["x"], t["w"], t["r"], residual_out=t["r"]), "r"),
    "norm fp8": (lambda t: afd.rms_norm(t["x"], t["w"], t["r"], dtype=F8, out=t["q"], out_scales=t["s"], residual_out=t["x"]), "q s x"),
    "norm, new memory": (lambda t: afd.rms_norm(t["x"], t["w"], t["r"], keep_rstd=True), ""),
    "norm_grad out": (lambda t: afd.rms_norm_grad(t["x"], t["r"], t["w"], t["rstd"], out=t["out"]), "out"),
    "norm_grad over grad": (lambda t: afd.rms_norm_grad(t["x"], t["r"], t["w"], t["rstd"], out=t["x"], weight_grad=False), "x"),
    "norm_grad, new memory": (lambda t: afd.rms_norm_grad(t["x"], t["r"], t["w"], t["rstd"]), ""),
    "route ids": (lambda t: afd.route_tokens(t["l"], 2, bias=t["bias"], live=t["live"], ids=t["ids"]), "ids"),
    "route weights": (lambda t: afd.route_tokens(t["l"], 2, weights=t["wt"]), "wt"),
    "route both": (lambda t: afd.route_tokens(t["l"], 2, ids=t["ids"], weights=t["wt"]), "ids wt"),
    "route, new memory": (lambda t: afd.route_tokens(t["l"], 2, bias=t["bias"]), ""),
    "route_grad out": (lambda t: afd.route_tokens_grad(t["wt"], t["l"], t["ids"], out=t["dl"]), "dl"),
    "route_grad, new memory": (lambda t: afd.route_tokens_grad(t["wt"], t["l"], t["ids"]), ""),
    "balance": (lambda t: afd.balance_loss(t["l"], t["ids"]), ""),
    "balance_grad out": (lambda t: afd.balance_loss_grad(t["g"], t["l"], t["ids"], t["slope"], out=t["dl"]), "dl"),
    "balance_grad, new memory": (lambda t: afd.balance_loss_grad(t["g"], t["l"], t["ids"], t["slope"]), ""),
}


@pytest.mark.parametrize("mode", [contextlib.nullcontext, torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("name", list(CALLS))
def test_given_outputs_are_written_in_autograds_sight(no_launch, name, mode):
    call, written = CALLS[name]
    t = _t()
    views = {k: v.detach() for k, v in t.items()}      # they share the counters
    before = {k: v._version for k, v in t.items()}
    with mode():
        call(t)
    for k, v in t.items():
        assert (v._version > before[k]) == (k in written.split()), k
        assert views[k]._version == v._version


def test_inference_tensors_have_no_counter(no_launch):
    with torch.inference_mode():
        t = _t()
        for call, _ in CALLS.values():
            call(t)


def test_a_saved_tensor_that_is_overwritten_is_found(no_launch):
    """torch's own products beside the calls, as a layer's projections are."""
    t = _t()
    p = torch.ones(256, dtype=BF, requires_grad=True)
    q = (t["r"] * p).sum()
    afd.rms_norm(t["x"], t["w"], t["r"], residual_out=t["r"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        q.backward()
    q = (t["wt"] * torch.ones(2, requires_grad=True)).sum()
    with torch.no_grad():
        afd.route_tokens(t["l"], 2, weights=t["wt"].detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        q.backward()
