"""GPU: what layer norm takes and refuses beyond its operands' shapes and types."""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu


def test_scratch_that_the_kernels_cannot_use_is_refused():
    x = torch.randn((50, 200), device="cuda")
    w = torch.ones(200, device="cuda")
    _, mean, rstd = gb.layer_norm(x, w)
    want = gb.layer_norm_backward(x, x, mean, rstd, w)
    nbytes = gb.load().gb_layer_norm_temp_bytes(50, 200)
    for temp in (torch.empty(nbytes, dtype=torch.uint8), torch.empty(nbytes, dtype=torch.uint8).pin_memory(),
                 torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            gb.layer_norm_backward(x, x, mean, rstd, w, temp=temp)
    with pytest.raises(gb.GbError):  # not 256-byte aligned
        gb.layer_norm_backward(x, x, mean, rstd, w, temp=torch.empty(nbytes + 1, dtype=torch.uint8, device="cuda")[1:])
    temp = torch.empty(nbytes // 4, device="cuda")  # of any type
    assert all(torch.equal(p, q) for p, q in zip(want, gb.layer_norm_backward(x, x, mean, rstd, w, temp=temp)))


def views(g, b, t, d, dtype):
    """Tensors of three and four dimensions whose rows have no one stride."""
    whole = torch.randn((b, t + 2, d + 8), generator=g).to(dtype).cuda()
    yield whole[:, 1:-1, :d]
    yield whole[:, 2:, 8:]
    yield torch.randn((t, b, d), generator=g).to(dtype).cuda().transpose(0, 1)
    yield torch.randn((b, 1, d), generator=g).to(dtype).cuda().expand(b, t, d)
    yield torch.randn((2, b, 3, d), generator=g).to(dtype).cuda().permute(1, 0, 2, 3)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 65])
def test_views_whose_leading_dimensions_do_not_merge(d, dt):
    g = torch.Generator().manual_seed(d)
    w, b = (torch.randn(d, generator=g).to(dt).cuda() for _ in range(2))
    for x in views(g, 3, 20, d, dt):
        dense = x.contiguous()
        want = gb.layer_norm(dense, w, b)
        got = gb.layer_norm(x, w, b)
        assert got[0].shape == x.shape and all(torch.equal(p, q) for p, q in zip(got, want))
        out = torch.empty_like(dense)
        assert gb.layer_norm(x, w, b, out=out)[0] is out and torch.equal(out, want[0])
        dy = torch.randn(x.shape, generator=g).to(dt).cuda()
        spread = torch.empty((*x.shape[:-2], x.shape[-2] + 1, d), dtype=dt, device="cuda")[..., 1:, :]
        spread.copy_(dy)
        wants = gb.layer_norm_backward(dy, dense, want[1], want[2], w)
        for args in ((dy, x), (spread, x), (spread, dense)):
            grads = gb.layer_norm_backward(*args, want[1], want[2], w)
            assert grads[0].shape == x.shape and all(torch.equal(p, q) for p, q in zip(grads, wants))
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        y, mean, rstd = gb.layer_norm(x, w, b, stream=s)
        grads = gb.layer_norm_backward(spread, x, mean, rstd, w, stream=s)
        s.synchronize()
        assert torch.equal(y, want[0]) and all(torch.equal(p, q) for p, q in zip(grads, wants))


def test_views_through_autograd():
    from stream_compaction_decoupled_gb300 import autograd
    g = torch.Generator().manual_seed(2)
    x = torch.randn((3, 9, 32), generator=g).cuda().requires_grad_()
    w = torch.randn(32, generator=g).cuda().requires_grad_()
    c = torch.randn((3, 8, 32), generator=g).cuda()
    got = torch.autograd.grad((autograd.layer_norm(x[:, 1:], w) * c).sum(), [x, w])
    want = torch.autograd.grad((autograd.layer_norm(x[:, 1:].contiguous(), w) * c).sum(), [x, w])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refused_shapes():
    x = torch.randn((3, 9, 32), device="cuda")
    _, mean, rstd = gb.layer_norm(x)
    for bad in (lambda: gb.layer_norm(x, out=torch.empty((3, 10, 32), device="cuda")[:, 1:]),
                lambda: gb.layer_norm(x.transpose(1, 2)),
                lambda: gb.layer_norm(x[:, 1:, ::2]),
                lambda: gb.layer_norm(torch.zeros((), device="cuda")),
                lambda: gb.layer_norm_backward(x[:, 1:], x, mean, rstd),
                lambda: gb.layer_norm_backward(x.transpose(1, 2), x, mean, rstd),
                lambda: gb.layer_norm_backward(x, x[:, 1:], mean, rstd)):
        with pytest.raises(ValueError):
            bad()
    assert gb.layer_norm(torch.zeros((0, 4, 32), device="cuda"))[0].shape == (0, 4, 32)
    assert gb.layer_norm(torch.zeros((2, 5, 32), device="cuda")[:, :0])[0].shape == (2, 0, 32)


@pytest.mark.parametrize("dweight", [True, False])
@pytest.mark.parametrize("dbias", [True, False])
def test_only_the_gradients_that_are_asked_for(monkeypatch, dweight, dbias):
    from stream_compaction_decoupled_gb300 import autograd, lm
    g = torch.Generator().manual_seed(3)
    x, w, b = (torch.randn(s, generator=g).cuda() for s in ((700, 96), (96,), (96,)))
    c = torch.randn((700, 96), generator=g).cuda()
    _, mean, rstd = gb.layer_norm(x, w, b)
    want = gb.layer_norm_backward(c, x, mean, rstd, w)
    got = gb.layer_norm_backward(c, x, mean, rstd, w, bias=dbias, dweight=dweight)
    for p, q, on in zip(got, want, (True, dweight, dbias)):
        assert torch.equal(p, q) if on else p is None
    seen = []
    whole = lm.layer_norm_backward
    monkeypatch.setattr(lm, "layer_norm_backward", lambda *a, **k: seen.append(k) or whole(*a, **k))
    leaves = [t.clone().requires_grad_(on) for t, on in ((x, True), (w, dweight), (b, dbias))]
    (autograd.layer_norm(*leaves) * c).sum().backward()
    assert seen == [{"bias": dbias, "dweight": dweight}]
    for t, q, on in zip(leaves, want, (True, dweight, dbias)):
        assert torch.equal(t.grad, q) if on else t.grad is None
    # A bias alone.
    leaves = [x.clone().requires_grad_(), b.clone().requires_grad_(dbias)]
    (autograd.layer_norm(leaves[0], None, leaves[1]) * c).sum().backward()
    assert torch.equal(leaves[1].grad, want[2]) if dbias else leaves[1].grad is None
    assert torch.equal(leaves[0].grad, gb.layer_norm_backward(c, x, mean, rstd)[0])
