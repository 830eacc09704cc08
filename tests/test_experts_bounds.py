"""What the network tests' bound of the second product would show: mistakes
planted in the reference lie outside it (CPU)."""
import pytest
import torch

from tests import experts_bounds as bounds
from tests import experts_ref as ref

CASES = [("bf16", 192, 0, 0), ("fp8", 384, 0, 0), ("bf16", 64, 4, 16), ("fp8", 128, 6, 8)]


def second(dtype, inner, S, rank):
    """The second product of a network over hidden rows rounded to its format."""
    counts, alpha, H = [15, 16, 17, 0, 31, 33, 1], 1, 256
    d = ref.make(7, len(counts), counts, alpha, inner, H, dtype, S=S, rank=rank)
    g = torch.Generator().manual_seed(3)
    h = torch.randn(d["rows"], inner, generator=g) * ref.silu(torch.randn(d["rows"], inner, generator=g))
    x, xs = ref.quant(h, 1) if dtype == "fp8" else (h.bfloat16(), None)
    return d, x, xs


@pytest.mark.parametrize("dtype,inner,S,rank", CASES)
def test_planted_mistakes_lie_outside_the_bound(dtype, inner, S, rank):
    d, x, xs = second(dtype, inner, S, rank)
    want, tol, live = bounds.product(d, x, xs, d["low"], d["w"], d["ws"])
    bound = ref.rounded(want, tol)

    def outside(got, rows=live):
        return float(((got - want).abs() > bound)[rows].double().mean())

    assert outside(torch.zeros_like(want)) > 0.98
    # 2 % of |y| exceed BF16's 0.4 % and the FP8 sums' 0.5 % of the values' size wherever
    # |y| is above 0.32 of it: three quarters of a normal distribution
    assert outside(want * 1.02) > 0.74
    w = d["w"].clone()
    w.view(torch.uint8).reshape(*w.shape[:2], -1)[..., : w.element_size()] = 0      # the first inner column dropped
    cut, _, _ = bounds.product(d, x, xs, d["low"], w, d["ws"])
    assert outside(cut) > 0.5
    if S:
        on = live & (d["tags"] >= 0) & (d["tags"] < S)
        bare, _, _ = bounds.product(d, x, xs, None, d["w"], d["ws"])
        assert outside(bare, on) > 0.95
        swapped = (d["low"][0].roll(1, 0), *d["low"][1:])
        other, _, _ = bounds.product(d, x, xs, swapped, d["w"], d["ws"])
        assert outside(other, on) > 0.95


def test_exponents_of_codes():
    q = torch.tensor([0.0, 2.0 ** -9, 2.0 ** -6, 0.03, -448.0, 1.875, -2.0]).to(torch.float8_e4m3fn).double()
    assert bounds.exponents(q).tolist() == [-float("inf"), -6, -6, -6, 8, 0, 1]
