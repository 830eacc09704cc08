"""A round's outputs and autograd on the GPU: memory that the caller gives to a round or
to the experts' calls, and that a graph saved, is found to be overwritten."""
import pytest
import torch

from tests import experts_ref as ref
from tests.test_gpu_experts import _dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, E, K, H, I, T, ALPHA = 1, 4, 2, 512, 256, 24, 16


def _afd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_layout_amd as afd
    return afd


def _rand(*shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).cuda()


def _experts(afd, F, dtype="bf16"):
    out = []
    for f in range(F):
        up = ref.make(31 + f, E // F, [1] * (E // F), 1, H, 2 * I, dtype, gated=True)
        down = ref.make(41 + f, E // F, [1] * (E // F), 1, I, H, dtype)
        out.append((afd.Experts(_dev(up["w"]), _dev(down["w"]), _dev(up["ws"]), _dev(down["ws"])), _dev(up["w"])))
    return out


def _found(loss):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("F", [1, 2])
def test_collected(F):
    """The norm of one round's sum, then the next round into the same memory."""
    afd = _afd()
    buf, experts = afd.Buffer(N, F, E, K, H, ALPHA, T), _experts(afd, F)
    x, ids, w = _rand(T, H, dtype=BF), torch.randint(0, E, (T, 1), generator=torch.Generator().manual_seed(1)).int(), _rand(T, K)
    ids = torch.cat([ids, (ids + 1) % E], 1).cuda()
    weight = torch.ones(H, device="cuda", requires_grad=True)

    def a_round(out, view=False):
        buf.source_dispatch(0, x, ids, w, bucket=T, out=out)
        for f, rec in enumerate([buf.worker_receive(f, bucket=T) for f in range(F)]):
            buf.worker_reply(f, buf.worker_experts(f, rec, experts[f][0]), rec.receipt)
        return buf.source_collect(0, view=view)

    out = torch.empty(T, H, dtype=BF, device="cuda")
    got = a_round(out)
    assert got is out
    loss = afd.rms_norm(got, weight).rows.float().sum()
    loss.backward(retain_graph=True)
    before = out._version
    buf.source_dispatch(0, x, ids, w, bucket=T, out=out)
    recs = [buf.worker_receive(f, bucket=T) for f in range(F)]
    replies = [buf.worker_experts(f, rec, experts[f][0]) for f, rec in enumerate(recs)]
    for f, rec in enumerate(recs):
        assert out._version == before         # not written yet: the graph stands
        buf.worker_reply(f, replies[f], rec.receipt)
    assert (out._version > before) == (F > 1)
    buf.source_collect(0)
    assert out._version > before
    _found(loss)
    loss, before = afd.rms_norm(got, weight).rows.float().sum(), out._version
    other = a_round(None)                     # new memory: the saved sum stands
    assert out._version == before and torch.equal(other, out) and other._version == 0
    loss.backward(retain_graph=True)
    with torch.no_grad():
        a_round(out)
    _found(loss)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_experts_outputs(dtype):
    afd = _afd()
    experts, up = _experts(afd, 1, dtype)[0]
    c = ref.make(3, E, [5] * E, 1, H, 2 * I, dtype, gated=True)
    x, xs = _dev(c["x"]), _dev(c["xs"])
    R, ends = c["rows"], torch.tensor(c["ends"], dtype=torch.int32).cuda()
    out = torch.zeros(R, H, dtype=BF, device="cuda")
    loss = (out * torch.ones(H, dtype=BF, device="cuda", requires_grad=True)).float().sum()
    afd.expert_ffn(x, ends, experts, x_scales=xs, out=out)
    _found(loss)
    out = torch.zeros(R, I, dtype=BF, device="cuda")
    loss = (out * torch.ones(I, dtype=BF, device="cuda", requires_grad=True)).float().sum()
    kw = dict(x_scales=xs, weight_scales=_dev(c["ws"]), activation="swiglu")
    afd.expert_product(x, ends, up, out=out, **kw)
    _found(loss)
    if dtype == "fp8":
        codes, scales = out.to(torch.float8_e4m3fn), torch.zeros(R, I // 128, device="cuda")
        before = codes._version, scales._version
        afd.expert_product(x, ends, up, out=codes, out_scales=scales, **kw)
        assert codes._version > before[0] and scales._version > before[1]
    with torch.inference_mode():
        afd.expert_ffn(x, ends, experts, x_scales=xs, out=torch.zeros(R, H, dtype=BF, device="cuda"))


def test_tags():
    afd = _afd()
    buf = afd.Buffer(N, 1, E, K, H, ALPHA, T)
    ids = (torch.arange(T * K).view(T, K) % E).int().cuda()
    buf.source_dispatch(0, _rand(T, H, dtype=BF), ids, _rand(T, K), bucket=T)
    rec = buf.worker_receive(0, bucket=T)
    out = torch.zeros(rec.receive_rows, dtype=torch.int32, device="cuda")
    before = out._version
    buf.worker_tags(0, [torch.arange(T, dtype=torch.int32, device="cuda")], rec, out=out)
    assert out._version > before
