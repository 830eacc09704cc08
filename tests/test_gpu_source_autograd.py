"""The source's calls and autograd on the GPU: what a recorded call saved and another
call then writes over is found by the backward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, H, E, K = 40, 256, 16, 4


def _afd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_layout_amd as afd
    return afd


def _rand(*shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).cuda()


def _asks(t):
    return t.clone().requires_grad_()


def _projection(afd):
    """A product that saves the stream; the next norm then adds to the stream in place."""
    stream, wq = _rand(T, H, dtype=BF), _asks(_rand(H, 32, dtype=BF))
    return (stream @ wq).sum(), lambda: afd.rms_norm(_rand(T, H, dtype=BF), _rand(H), stream, residual_out=stream)


def _norm_of_x(afd):
    x, w = _rand(T, H, dtype=BF), _asks(_rand(H))
    return afd.rms_norm(x, w).rows.float().sum(), lambda: afd.rms_norm(_rand(T, H, dtype=BF) + 1, _rand(H), out=x)


def _norm_of_the_stream(afd):
    """With only the weight asking, the stream that the call returns is what it saved."""
    n = afd.rms_norm(_rand(T, H, dtype=BF), _asks(_rand(H)), _rand(T, H, dtype=BF))
    assert not n.residual.requires_grad
    return n.rows.float().sum(), lambda: afd.rms_norm(_rand(T, H, dtype=BF), _rand(H), n.residual, residual_out=n.residual)


def _norm_by_its_gradient(afd):
    x, w = _rand(T, H, dtype=BF), _asks(_rand(H))
    y, h = _rand(T, H, dtype=BF), _rand(T, H, dtype=BF)
    return afd.rms_norm(x, w).rows.float().sum(), lambda: afd.rms_norm_grad(y, h, w.detach(), torch.ones(T, device="cuda"), out=x)


def _routes_of_logits(afd):
    l = _asks(_rand(T, E))
    ids = afd.route_tokens(_rand(T, E), K).ids
    r = afd.route_tokens(l, K)
    return r.weights.sum(), lambda: afd.route_tokens_grad(_rand(T, K), _rand(T, E), ids, out=l.detach())


def _routes_ids(afd):
    r = afd.route_tokens(_asks(_rand(T, E)), K)
    return r.weights.sum(), lambda: afd.route_tokens(_rand(T, E), K, ids=r.ids)


def _balance_of_logits(afd):
    l = _asks(_rand(T, E))
    ids = afd.route_tokens(l.detach(), K).ids
    slope = torch.ones(E, device="cuda")
    return afd.balance_loss(l, ids).loss, lambda: afd.balance_loss_grad(slope[0].clone(), _rand(T, E), ids, slope, out=l.detach())


def _balance_ids(afd):
    """The next batch's routes in the buffer of the last one's."""
    l, ids = _asks(_rand(T, E)), torch.empty(T, K, dtype=torch.int32, device="cuda")
    afd.route_tokens(l.detach(), K, ids=ids)
    return afd.balance_loss(l, ids).loss, lambda: afd.route_tokens(_rand(T, E), K, ids=ids)


def _weights(afd):
    w = torch.empty(T, K, device="cuda")
    afd.route_tokens(_rand(T, E), K, weights=w)
    return (w * _asks(_rand(K))).sum(), lambda: afd.route_tokens(_rand(T, E) * 2, K, weights=w)


def _source_norm(afd):
    buf = afd.Buffer(1, 1, E, K, H, capacity=T)
    stream, wq = _rand(T, H, dtype=BF), _asks(_rand(H, 32, dtype=BF))
    return (stream @ wq).sum(), lambda: buf.source_norm(0, _rand(T, H, dtype=BF), _rand(H), stream, residual_out=stream)


CASES = [_projection, _norm_of_x, _norm_of_the_stream, _norm_by_its_gradient, _routes_of_logits, _routes_ids, _balance_of_logits,
         _balance_ids, _weights, _source_norm]


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_a_saved_tensor_that_is_overwritten_is_found(case, off):
    afd = _afd()
    loss, over = case(afd)
    loss.backward(retain_graph=True)          # whole before, refused behind
    with torch.set_grad_enabled(not off):
        over()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_graphs_of_new_memory_stand():
    """Calls that make their own outputs, and outputs that no graph saved, disturb no graph."""
    afd = _afd()
    x, w, l = _asks(_rand(T, H, dtype=BF)), _asks(_rand(H)), _asks(_rand(T, E))
    n, r = afd.rms_norm(x, w, x), afd.route_tokens(l, K)
    b = afd.balance_loss(l, r.ids)
    with torch.no_grad():
        other = afd.rms_norm(x, w, x, residual_out=torch.empty_like(x), out=torch.empty_like(x))
        again = afd.route_tokens(l, K, ids=torch.empty_like(r.ids))
    (n.rows.float().sum() + r.weights.sum() + b.loss).backward()
    assert x.grad is not None and l.grad is not None
    assert torch.equal(other.residual, n.residual) and torch.equal(again.ids, r.ids)


def _negated(t):
    """t as the imaginary part of a conjugate: its sign stands beside the memory."""
    n = torch.complex(torch.zeros_like(t), -t).conj().imag
    assert n.is_neg() and torch.equal(n, t)
    return n


def test_a_gradient_whose_sign_is_not_in_memory():
    """Gradients that pass a complex number arrive with their sign held back."""
    afd = _afd()
    l = _asks(_rand(T, E))
    with torch.no_grad():
        r = afd.route_tokens(l, K)
        b = afd.balance_loss(l, r.ids)
        want = afd.balance_loss_grad(torch.full((), 2.0, device="cuda"), l, r.ids, b.slope)
    seen = []
    loss = afd.balance_loss(l, r.ids).loss
    loss.register_hook(lambda g: seen.append(g.is_neg()))
    (torch.complex(torch.ones_like(loss), loss).conj() * (1 + 2j)).real.backward()     # the loss times 2
    assert seen == [True]
    assert torch.equal(l.grad, want)
    assert torch.equal(afd.balance_loss_grad(_negated(torch.full((), 2.0, device="cuda")), l.detach(), r.ids, b.slope), want)
    # every element of the weights' gradient, and a gradient of one element, which any stride makes contiguous
    for tokens, k in ((T, K), (1, 1)):
        x, g = l.detach()[:tokens].requires_grad_(), _rand(tokens, k)
        ids = afd.route_tokens(x.detach(), k, renormalize=False).ids
        (d,) = torch.autograd.grad(afd.route_tokens(x, k, renormalize=False).weights, x, _negated(g))
        assert torch.equal(d, afd.route_tokens_grad(g, x.detach(), ids, renormalize=False))
    assert torch.equal(afd.route_tokens_grad(_negated(g), x.detach(), ids, renormalize=False), d)
    x, w, r = _asks(_rand(T, H)), _asks(_rand(H)), _asks(_rand(T, H))
    n = afd.rms_norm(x, w, r)
    grad = _rand(T, H)
    (d,) = torch.autograd.grad(n.residual, x, _negated(grad))
    assert torch.equal(d, grad)


def test_one_expert_whose_sign_is_not_in_memory():
    """Logits of one expert, which any stride lets pass: refused at every call, as before and behind those
    of the same layout that are taken."""
    afd = _afd()
    l, ids, one = _rand(T, 1), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones((), device="cuda")
    b, dw, slope = torch.full((1,), 0.25, device="cuda"), _rand(T, 1), torch.ones(1, device="cuda")
    wide = torch.empty(T, 2, device="cuda")[:, :1].copy_(l)
    kw = dict(scoring="sigmoid", renormalize=False)
    for _ in range(2):
        x = _negated(l)
        for call in (lambda: afd.route_tokens(x, 1, **kw), lambda: afd.route_tokens(l, 1, bias=_negated(b), **kw),
                     lambda: afd.route_tokens(x.detach().requires_grad_(), 1, **kw), lambda: afd.route_tokens_grad(dw, x, ids, **kw),
                     lambda: afd.balance_loss(x, ids), lambda: afd.balance_loss_grad(one, x, ids, slope),
                     lambda: afd.balance_loss_grad(one, l, ids, _negated(slope))):
            with pytest.raises(ValueError, match="resolve_neg"):
                call()
        r = afd.route_tokens(x.resolve_neg(), 1, bias=b, **kw)
        for y in (l, wide):
            assert torch.equal(afd.route_tokens(y, 1, bias=b, **kw).weights, r.weights)
            afd.balance_loss_grad(one, y, ids, afd.balance_loss(y, ids).slope)
            afd.route_tokens_grad(dw, y, ids, **kw)
