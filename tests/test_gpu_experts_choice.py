"""The experts' calls with every expected number of rows per expert: whichever
kernel that chooses, the values are right."""
import pytest
import torch

from tests import experts_bounds as bounds
from tests import experts_ref as ref
from tests.test_gpu_experts import COUNTS, FILL, _afd, _dev, _low, _print
from tests.test_gpu_experts_network import ARENA, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("each", [0, 1, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,k,n,S", [("bf16", 320, 144, 0), ("fp8", 384, 272, 0), ("bf16", 192, 80, 3), ("fp8", 128, 144, 3)])
@pytest.mark.parametrize("rows", [0, ARENA])
def test_any_expectation_gives_right_values(each, dtype, k, n, S, rows):
    afd = _afd()
    _print("expected rows", each, dtype, k, n, S, rows)
    counts, alpha = COUNTS["edges"]
    c = ref.make(19, len(counts), counts, alpha, k, n, dtype, S=S, rank=8 if S else 0)
    R = max(rows, c["rows"])
    out = torch.full((R, n), FILL, dtype=torch.bfloat16, device="cuda")
    afd.expert_product(_wide(c["x"], R, 0x7F if dtype == "fp8" else float("nan")), torch.tensor(c["ends"], dtype=torch.int32).cuda(),
                       _dev(c["w"]), alignment=alpha, x_scales=_wide(c["xs"], R, 1.0), weight_scales=_dev(c["ws"]),
                       adapters=_low(afd, c["low"]), row_adapters=_wide(c["tags"], R, 0), out=out, rows_per_expert=each)
    want, tol, live = bounds.product(c, c["x"], c["xs"], c["low"], c["w"], c["ws"])
    got = out.double().cpu()
    assert (got[c["rows"]:] == FILL).all() and (got[:c["rows"]][~live] == FILL).all()
    assert ((got[:c["rows"]] - want).abs() <= ref.rounded(want, tol))[live].all()


def test_expectations_refused():
    afd = _afd()
    x, ends = torch.zeros((8, 64), device="cuda").bfloat16(), torch.tensor([8], dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 16, 64), device="cuda").bfloat16()
    ex = afd.Experts(torch.zeros((1, 128, 64), device="cuda").bfloat16(), torch.zeros((1, 64, 64), device="cuda").bfloat16())
    for bad in (-1, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            afd.expert_product(x, ends, w, rows_per_expert=bad)
        with pytest.raises(ValueError):
            afd.expert_ffn(x, ends, ex, rows_per_expert=bad)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_rounds_with_host_counts(dtype):
    """worker_experts on rows that the host counted (exact, with their alignment's
    padding): the rows of a round without host counts, within the sums' orders."""
    afd = _afd()
    _print("host counts", dtype)
    N, F, E, K, H, inner, alpha, T = 2, 2, 16, 4, 256, 128, 128, 200
    g = torch.Generator().manual_seed(21)
    u = ref.make(22, E // F, [1] * (E // F), 1, H, 2 * inner, dtype, gated=True)
    d = ref.make(23, E // F, [1] * (E // F), 1, inner, H, dtype)
    ex = afd.Experts(_dev(u["w"]), _dev(d["w"]), _dev(u["ws"]), _dev(d["ws"]))
    buf = afd.Buffer(N, F, E, K, H, alpha, T, dtype)
    x = torch.randn(N, T, H, generator=g)
    ids = torch.stack([torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) for _ in range(N)]).int().cuda()
    for counted in (False, True):
        for s in range(N):
            q, qs = ref.quant(x[s], 1) if dtype == "fp8" else (x[s].bfloat16(), None)
            buf.source_dispatch(s, _dev(q), ids[s].contiguous(), torch.ones(T, K, device="cuda"), _dev(qs), bucket=T,
                                read_host_counts=counted)
        for f in range(F):
            rec = buf.worker_receive(f, bucket=T, read_host_counts=counted)
            ends = rec.ends.tolist()
            assert (rec.receive_rows == -(-ends[-1] // alpha) * alpha) == counted
            got = buf.worker_experts(f, rec, ex)
            n = ends[-1]
            xq = rec.rows.view(torch.uint8).cpu().view(torch.float8_e4m3fn)[:n] if dtype == "fp8" else rec.rows.cpu()[:n]
            want, tol, live = ref.run_ffn(xq, rec.scales.cpu()[:n] if dtype == "fp8" else None, u["w"], u["ws"], d["w"], d["ws"],
                                          None, None, None, ends, alpha, n)
            assert ((got.double().cpu()[:n] - want).abs() <= ref.rounded(want, tol))[live].all()
            buf.worker_reply(f, got, rec.receipt)
        for s in range(N):
            buf.source_collect(s)
