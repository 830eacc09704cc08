"""Route weights and their gradients where logits lie far apart: bounds that do not grow
with the distance.  In U, half a float32 step, relative to the value:

an exponential is 3 off (its instruction a step, the correction of its argument one
rounding), a reciprocal of 1 + z 4 (z's own error counts 1.5 at most, as z falls faster than
it grows; the sum, Newton's step with a margin), a sum of chosen terms 6 more than a term (two
slots, then up to 64 lanes), a division 1, the scale 1."""
import pytest
import torch

from tests import source_ref as ref
from tests.test_gpu_source import BF, F32, _afd, _gen, _print, _rand

pytestmark = pytest.mark.gpu

# a softmax over the chosen: term, sum of terms, division, scale; over all: the sum is of 512 terms
# at most, 13 additions deep, whose own distances x cost 2.3 x each, 9 on the mean, beside 2 for the
# instruction; sigmoids: term 3, reciprocal 4, product 1, and the sum and division where renormalised
BOUND = {("softmax", True): 3 + 3 + 6 + 1 + 1, ("softmax", False): 3 + 9 + 2 + 13 + 1 + 1 + 1,
         ("sigmoid", True): 8 + 8 + 6 + 1 + 1, ("sigmoid", False): 3 + 4 + 1 + 1}
LEFT = 3 + 4 + 1      # 1 - sigmoid


def _far(seed, T, E, dtype, shift):
    """Logits spread evenly over 80 below a largest one near `shift`."""
    g = _gen(seed)
    l = -80 * torch.rand((T, E), generator=g) + shift
    l[:, 0] = shift
    return l.to(dtype)


@pytest.mark.parametrize("E,K", [(8, 8), (32, 32), (64, 20), (100, 32), (200, 32), (300, 32), (512, 32)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("shift", [0.0, 1.3, 40.0, 81.0])
def test_weights_of_far_logits(E, K, dtype, scoring, renormalize, shift):
    afd = _afd()
    _print("far", E, K, dtype, scoring, renormalize, shift)
    T = 200
    l = _far(E + K, T, E, dtype, shift)
    # the far ones are chosen too: a bias that lifts every other expert
    b = torch.zeros(E)
    b[::2] = 2.0
    for bias in (None, b):
        r = afd.route_tokens(l.cuda(), K, scoring=scoring, renormalize=renormalize, scale=1.5,
                             bias=None if bias is None else bias.cuda())
        ids = r.ids.cpu().long()
        w, _ = ref.weights(l, ids, scoring, renormalize, 1.5)
        tol = BOUND[scoring, renormalize] * ref.U * w.abs() + 2 * ref.TINY
        ref.check(r.weights, w, tol, "weights")


@pytest.mark.parametrize("E,K", [(8, 8), (100, 32), (200, 32), (512, 32)])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("shift", [0.0, 40.0, 81.0])
def test_sigmoids_gradient_of_far_logits(E, K, renormalize, shift):
    afd = _afd()
    T = 200
    l = _far(E, T, E, F32, shift)
    g = _gen(5)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    dw = _rand(g, T, K)
    d = afd.route_tokens_grad(dw.cuda(), l.cuda(), ids.int().cuda(), scoring="sigmoid", renormalize=renormalize)
    w, _ = ref.weights(l, ids, "sigmoid", renormalize, 1.0)
    left = torch.sigmoid(-torch.take_along_dim(l.double(), ids, 1))
    dot, size = ((dw.double() * w).sum(1, keepdim=True), (dw.double() * w).abs().sum(1, keepdim=True))
    if not renormalize:
        dot, size = torch.zeros_like(dot), torch.zeros_like(dot)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, w * left * (dw.double() - dot))
    one = BOUND["sigmoid", renormalize]
    # the weight, the sum of its products with the gradients (one rounding, six additions), the
    # difference, two products and the factor 1 - sigmoid
    n = one + (one + 1 + 6 + 1 if renormalize else 1) + 2 + LEFT
    tol = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, n * ref.U * w * left * (dw.double().abs() + size))
    ref.check(d, want, tol + 2 * ref.TINY * (1 + dw.abs().amax(1, keepdim=True).double()), "dlogits")
