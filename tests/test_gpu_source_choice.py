"""The biased choice far from zero, where many scores are equal or nearly so: by the
64-bit sums themselves, place by place."""
import pytest
import torch

from tests import source_ref as ref
from tests.test_gpu_source import BF, F32, INF, NAN, _afd, _gen, _logits, _print, _rand

pytestmark = pytest.mark.gpu

# Two 64-bit evaluations of a score (at most 1) differ by an exponential's step, a sum of up to
# 512 terms in another order (some 14 roundings of one and as many of the other) and a division:
# below 64 half steps of 1.  The sums with the bias (at most 4) add one half step of 4 each.
NEAR = 2.0 ** -46


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,K", [(8, 4), (64, 32), (128, 8), (250, 9), (256, 8), (300, 32), (500, 12)])
@pytest.mark.parametrize("odd", [False, True])
def test_choice_far_from_zero(scoring, dtype, E, K, odd):
    afd = _afd()
    _print("far choice", scoring, dtype, E, K, odd)
    g = _gen(E + K)
    l = torch.cat([_logits(g, 16, E, F32) + 300, _logits(g, 16, E, F32) * 40, _logits(g, 16, E, F32) - 300,
                   _logits(g, 16, E, F32) * 4 + 36]).to(dtype)
    b = (_rand(g, E, std=0.2) * 8).round() / 8
    if odd:
        b[0], b[5 % E], b[6 % E] = -INF, NAN, INF
    ids = afd.route_tokens(l.cuda(), K, scoring=scoring, bias=b.cuda()).ids.cpu().long()
    want = ref.choose(l, K, scoring, b, None)
    assert torch.equal(ids >= 0, want >= 0)
    score, on = ref.scores(l, scoring), ids >= 0
    key = score + b.double()
    got, top = (torch.take_along_dim(key, i.clamp(min=0), 1) for i in (ids, want))
    assert (((got - top).abs() <= NEAR) | (got == top) | ~on).all()
    for row in range(len(l)):
        chosen = ids[row][on[row]].tolist()
        assert len(set(chosen)) == len(chosen)
        # keys that no error of the score moves: where all that are near to a place's are of these
        # and equal to it, the lowest id that is left has the place
        lo, hi = (score[row] * (1 + s * 2.0 ** -46) + b.double() for s in (-1, 1))
        sure = lo == hi
        for k in range(len(chosen)):
            near = ((key[row] - top[row, k]).abs() <= 2 * NEAR) | (key[row] == top[row, k])
            if sure[near].all() and (key[row][near] == top[row, k]).all():
                assert ids[row, k] == want[row, k], (row, k)
