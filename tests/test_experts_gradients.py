"""The experts' calls are forward calls: whatever asks for a gradient, or
carries a forward one, is refused before anything else (so these run on host
tensors, which are refused later)."""
import pytest
import torch
from torch.autograd import forward_ad

import combine_layout_amd as afd

X, ENDS = torch.zeros(4, 128), torch.tensor([4], dtype=torch.int32)
W, SCALE, ONE = torch.zeros(1, 128, 128), torch.ones(1, 1, 1), torch.ones(4, 1)
LOW = afd.LowRank(torch.zeros(2, 1, 8, 128), torch.zeros(2, 1, 128, 8), torch.ones(2))
EXPERTS = object()      # not looked at before the refusal


def asks(t):
    return t.clone().requires_grad_()


def calls(mark):
    """Every call with one of its tensors marked."""
    product, ffn = afd.expert_product, afd.expert_ffn
    for i in range(3):
        low = LOW._replace(**{LOW._fields[i]: mark(LOW[i])})
        yield f"product {LOW._fields[i]}", lambda low=low: product(X, ENDS, W, adapters=low)
        yield f"network up {LOW._fields[i]}", lambda low=low: ffn(X, ENDS, EXPERTS, adapters=afd.ExpertAdapters(low, LOW))
        yield f"network down {LOW._fields[i]}", lambda low=low: ffn(X, ENDS, EXPERTS, adapters=afd.ExpertAdapters(LOW, low))
    yield "product x", lambda: product(mark(X), ENDS, W)
    yield "product weight", lambda: product(X, ENDS, mark(W))
    yield "product x_scales", lambda: product(X, ENDS, W, x_scales=mark(ONE))
    yield "product weight_scales", lambda: product(X, ENDS, W, weight_scales=mark(SCALE))
    yield "product out", lambda: product(X, ENDS, W, out=mark(X))
    yield "product out_scales", lambda: product(X, ENDS, W, out_scales=mark(ONE))
    yield "network x", lambda: ffn(mark(X), ENDS, EXPERTS)
    yield "network x_scales", lambda: ffn(X, ENDS, EXPERTS, x_scales=mark(ONE))
    yield "network out", lambda: ffn(X, ENDS, EXPERTS, out=mark(X))
    yield "pack_weights", lambda: afd.pack_weights(mark(W))
    packed = afd.PackedWeights(W, W.shape, W.dtype)
    yield "Experts up", lambda: afd.Experts(mark(W), packed)
    yield "Experts down", lambda: afd.Experts(packed, mark(W))
    yield "Experts up_scales", lambda: afd.Experts(packed, packed, mark(SCALE), SCALE)
    yield "Experts down_scales", lambda: afd.Experts(packed, packed, SCALE, mark(SCALE))


@pytest.mark.parametrize("what,call", list(calls(asks)))
def test_what_asks_for_a_gradient_is_refused(what, call):
    with pytest.raises(ValueError, match="gradients"):
        call()


def test_without_gradients_it_is_a_plain_tensor():
    packed = afd.PackedWeights(W, W.shape, W.dtype)
    with torch.no_grad():
        e = afd.Experts(packed, packed, asks(SCALE), asks(SCALE))
        with pytest.raises(ValueError, match="contiguous"):      # of the host tensor
            afd.expert_product(asks(X), ENDS, asks(W))
    assert not e.up_scales.requires_grad and not e.down_scales.requires_grad
    with pytest.raises(ValueError, match="contiguous"):
        afd.pack_weights(W)


def test_dual_tensors_are_refused():
    with forward_ad.dual_level():
        for grad in (False, True):
            with torch.set_grad_enabled(grad):
                for what, call in calls(lambda t: forward_ad.make_dual(t, torch.ones_like(t))):
                    with pytest.raises(ValueError, match="gradients"):
                        call()
        with pytest.raises(ValueError, match="contiguous"):      # the primals inside a level are plain tensors
            afd.expert_product(X, ENDS, W)
