"""The linear layer, dropout and the join as programs use them: autograd wrappers and modules against the same calls made by
hand, bit for bit; views; what the loss does not use; a generator that is advanced in between; a decoder's steps served,
eager and captured; a training step of several layers in a graph."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_ffn_03_amd import autograd as ag
from activation_sparse_ffn_03_amd import twell as tw
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)


def _leaf(t):
    return t.detach().clone().requires_grad_()


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("bias,res", [(None, None), (F32, BF), (BF, F32)])
def test_linear_autograd(act, bias, res):
    require_gpu()
    rnd = _rnd(1)
    x, w = _leaf(rnd(3, 50, 200, dtype=BF)), _leaf(rnd(129, 200, dtype=BF, scale=0.1))
    b = None if bias is None else _leaf(rnd(129, dtype=bias))
    r = None if res is None else _leaf(rnd(3, 50, 129, dtype=res))
    y = ag.linear(x, w, b, act, r, F32)
    g = rnd(3, 50, 129)
    y.backward(g)
    x2, pre = x.detach().reshape(150, 200), torch.empty(150, 129, dtype=BF, device="cuda")
    want = tw.linear(x2, w.detach(), bias=None if b is None else b.detach(), act=act, dtype=F32, pre=pre,
                     residual=None if r is None else r.detach().reshape(150, 129))
    assert torch.equal(y.detach().reshape(150, 129), want)
    d = tw.linear_bwd(g.reshape(150, 129), x2, w.detach(), act=act, pre=pre, dx_dtype=BF, dw_dtype=BF)
    assert torch.equal(x.grad.reshape(150, 200), d.dx) and torch.equal(w.grad, d.dw)
    if b is not None:
        assert b.grad.dtype == bias and torch.equal(b.grad, d.db.to(bias))
    if r is not None:
        assert torch.equal(r.grad, g.to(res))


def test_linear_of_which_not_all_is_trained_and_views():
    require_gpu()
    rnd = _rnd(2)
    flat = rnd(1 + 40 * 97, dtype=BF)
    x = flat[1:].view(40, 97)  # begins at two bytes
    w = rnd(60, 97, dtype=BF)
    assert torch.equal(ag.linear(x, w), tw.linear(x.clone(), w))
    for train in ((True, False, False), (False, True, False), (False, False, True)):
        leaves = [_leaf(t) if k else t for t, k in zip((x, w, rnd(60)), train)]
        ag.linear(leaves[0], leaves[1], leaves[2], "silu").float().square().sum().backward()
        assert [t.grad is not None for t in leaves] == list(train)
    wt = _leaf(rnd(97, 60, dtype=BF))
    ag.linear(x, wt.t(), act="relu").sum().backward()  # a transposed weight
    assert wt.grad.shape == (97, 60)
    with pytest.raises(ValueError, match="residual"):
        ag.linear(x, w, residual=rnd(1, 60, dtype=BF))
    with pytest.raises(TypeError, match="bfloat16"):
        ag.linear(x.float(), w)
    with torch.no_grad():
        assert not ag.linear(leaves[0], leaves[1], leaves[2]).requires_grad


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_autograd_with_a_generator_that_is_advanced(dtype):
    require_gpu()
    rnd = _rnd(3)
    rng = tw.make_rng(11, 5)
    x = _leaf(rnd(4, 30, 77, dtype=dtype))
    y = ag.dropout(x, rng, 0.3, site=2)
    rng[1] += 1
    g = rnd(4, 30, 77, dtype=dtype)
    y.backward(g)
    old = tw.make_rng(11, 5)
    assert torch.equal(y.detach().view(120, 77), tw.dropout(x.detach().view(120, 77), old, 0.3, site=2))
    assert torch.equal(x.grad.view(120, 77), tw.dropout(g.view(120, 77), old, 0.3, site=2))
    assert not torch.equal(y, ag.dropout(x, rng, 0.3, site=2))


def _join_by_hand(r, y, w, pw, gate, alpha, p, rng, site, d_res, d_out):
    f = tw.join_rms_norm(r, y, w, post_weight=pw, gate=gate, alpha=alpha, eps=EPS, p=p, rng=rng, site=site, stats=True)
    g = tw.join_rms_norm_bwd(d_out, f.residual, f.rstd, y, w, post_weight=pw, post_rstd=f.post_rstd, gate=gate, alpha=alpha, p=p,
                             rng=rng, site=site, d_residual=d_res)
    return f, g


@pytest.mark.parametrize("used", ["both", "stream", "norm"])
@pytest.mark.parametrize("post,gate_rows,p", [(True, 0, 0.2), (True, 3, 0.0), (False, 1, 0.1), (False, 0, 0.0)])
def test_join_autograd(used, post, gate_rows, p):
    require_gpu()
    rnd = _rnd(4)
    B, T, D = 3, 20, 250
    r, y, w = _leaf(rnd(B, T, D, dtype=BF)), _leaf(rnd(B, T, D)), _leaf(1 + rnd(D, dtype=BF, scale=0.1))
    pw = _leaf(1 + rnd(D, dtype=BF, scale=0.1)) if post else None
    gate = None if gate_rows == 0 else _leaf(rnd(D, dtype=BF) if gate_rows == 1 else rnd(gate_rows, D))
    rng = tw.make_rng(1, 2)
    st, out = ag.join_rms_norm(r, y, w, pw, gate, 0.9, EPS, p, rng, 3)
    rng[1] += 7
    ds, dn = rnd(B, T, D, dtype=BF), rnd(B, T, D, dtype=BF)
    torch.autograd.backward([t for t, k in ((st, "stream"), (out, "norm")) if used in (k, "both")],
                            [t for t, k in ((ds, "stream"), (dn, "norm")) if used in (k, "both")])
    d = [None if t is None else t.detach() for t in (w, pw, gate)]
    f, g = _join_by_hand(r.detach().view(-1, D), y.detach().view(-1, D), *d, 0.9, p, tw.make_rng(1, 2), 3,
                         ds.view(-1, D) if used != "norm" else None, dn.view(-1, D) if used != "stream" else torch.zeros(B * T, D, dtype=BF, device="cuda"))
    assert torch.equal(st.detach().view(-1, D), f.residual) and torch.equal(out.detach().view(-1, D), f.out)
    assert torch.equal(r.grad.view(-1, D), g.dr) and torch.equal(y.grad.view(-1, D), g.dy)
    assert torch.equal(w.grad, g.dw.to(BF))
    if post:
        assert torch.equal(pw.grad, g.dpost.to(BF))
    if gate is not None:
        assert torch.equal(gate.grad, g.dgate.to(gate.dtype))


def test_join_takes_views_and_refuses_what_does_not_fit():
    require_gpu()
    rnd = _rnd(5)
    r, y, w = rnd(31 * 99 + 1, dtype=BF)[1:].view(31, 99), rnd(99, 31).t(), rnd(100)[1:]
    st, out = ag.join_rms_norm(r, y, w)
    want = tw.join_rms_norm(r.clone(), y.contiguous(), w.clone())
    assert torch.equal(st, want.residual) and torch.equal(out, want.out)
    with pytest.raises(ValueError, match="divides 31"):
        ag.join_rms_norm(r, y, w, gate=rnd(2, 99))
    with pytest.raises(ValueError, match="rng"):
        ag.join_rms_norm(r, y, w, p=0.1)
    with pytest.raises(ValueError, match="shape of the residual"):
        ag.join_rms_norm(r, y[:1], w)


def test_modules_hold_what_they_say():
    require_gpu()
    ffn = ag.TwellDenseFFN(256, 640, "gelu")
    assert [tuple(p.shape) for p in ffn.parameters()] == [(640, 256), (640,), (256, 640), (256,)]
    rnd = _rnd(6)
    x, r = rnd(5, 7, 256, dtype=BF), rnd(5, 7, 256, dtype=BF)
    h = tw.linear(x.view(35, 256), ffn.up.weight.detach(), bias=ffn.up.bias.detach(), act="gelu")
    want = tw.linear(h, ffn.down.weight.detach(), bias=ffn.down.bias.detach(), residual=r.view(35, 256))
    assert torch.equal(ffn(x, r).detach().view(35, 256), want)
    ffn(x, r).float().square().mean().backward()
    assert all(p.grad is not None and bool(p.grad.isfinite().all()) for p in ffn.parameters())
    join = ag.TwellJoin(256, gate=0.5, alpha=0.8, p=0.3, site=4)
    rng = tw.make_rng(3)
    st, _ = join(x, r, rng)
    by_hand = lambda p: tw.join_rms_norm(x.view(35, 256), r.view(35, 256), join.weight.detach(), post_weight=join.post_weight.detach(),  # noqa: E731
                                         gate=join.gate.detach(), alpha=0.8, eps=EPS, p=p, rng=rng, site=4)
    assert torch.equal(st.detach().view(35, 256), by_hand(0.3).residual)
    join.eval()
    assert torch.equal(join(x, r)[0].detach().view(35, 256), by_hand(0.0).residual)
    with pytest.raises(ValueError, match="act"):
        ag.TwellLinear(8, 8, act="tanh")


def test_block_with_a_join_trains():
    """Stream, a dense layer whose output is joined with dropout, the sparse block behind it: gradients of every parameter, the
    join's the ones that the calls by hand give."""
    require_gpu()
    torch.manual_seed(0)
    D, F, N = 128, 512, 96
    block = ag.TwellBlock(D, F, cfg=ag.TwellConfig(tile_n=64, slots=64, row_cap=512, ovf_frac=1.0, dense_frac=1.0),
                          join=ag.TwellJoin(D, gate=0.7, p=0.1, site=1))
    dense = ag.TwellLinear(D, D, act="silu")
    rng = tw.make_rng(9)
    rnd = _rnd(7)
    stream = _leaf(rnd(N, D, dtype=BF))
    delta = dense(stream)
    st, y = block(stream, delta, torch.full((N,), 0.8, device="cuda"), rng)
    (st.float().square().mean() + y.square().mean()).backward()
    for name, p in list(block.named_parameters()) + list(dense.named_parameters()):
        assert p.grad is not None and bool(p.grad.isfinite().all()) and bool((p.grad != 0).any()), name
    want = tw.join_rms_norm(stream.detach(), delta.detach(), block.norm.weight.detach(), post_weight=block.norm.post_weight.detach(),
                            gate=block.norm.gate.detach(), p=0.1, rng=rng, site=1)
    assert torch.equal(st.detach(), want.residual)
    with pytest.raises(ValueError, match="join"):
        block(stream)


@pytest.mark.parametrize("gate", ["bf16", "fp8", "mx4"])
def test_serving_with_norms_on_both_sides(gate):
    """A decoder's steps: y of one call is the delta of the next, joined behind a norm with a channel gate and a scaled residual;
    the eager calls against the join and the block by hand, captured ones against the eager."""
    require_gpu()
    N, D, F = 4, 512, 1024
    rnd = _rnd(8)
    dims = tw.make_dims(N, D, F, 64, 64, 0, 8, 0)
    w = rnd(F, D, dtype=BF, scale=D ** -0.5)
    w = {"bf16": lambda: w, "fp8": lambda: tw.quantize_e4m3(w), "mx4": lambda: tw.quantize_mx4(w)}[gate]()
    nw, up, down = (1 + rnd(D, scale=0.2)).to(BF), rnd(F, D, dtype=BF, scale=D ** -0.5), rnd(F, D, dtype=BF, scale=F ** -0.5)
    t = torch.full((N,), 1.15, device="cuda")
    join = dict(post_weight=(1 + rnd(D, scale=0.2)).to(BF), layer_gate=rnd(D, dtype=BF), alpha=0.9)
    stream, delta = rnd(N, D, dtype=BF), rnd(N, D)
    serve, plain, eager = (tw.TwellServe(dims, gate, EPS) for _ in range(3))
    by_hand = stream.clone()
    y = serve.forward(stream, delta, nw, w, up, down, t, **join)
    j = tw.join_rms_norm(by_hand, delta, nw, post_weight=join["post_weight"], gate=join["layer_gate"], alpha=0.9, eps=EPS,
                         out=tw.JoinOut(by_hand, None, None, None, torch.empty(N, device="cuda"), None))
    want = plain.forward(j.residual, None, nw, w, up, down, t)
    assert torch.equal(stream, by_hand) and torch.equal(y, want)
    want_stream = stream.clone()
    eager.y.copy_(y)
    graph = serve.capture(stream, y, nw, w, up, down, t, **join)
    want = eager.y
    for _ in range(3):
        graph.replay()
        want = eager.forward(want_stream, want, nw, w, up, down, t, **join)
        torch.cuda.synchronize()
        assert torch.equal(stream, want_stream) and torch.equal(y, want)
    for bad in (dict(post_weight=nw), dict(layer_gate=nw), dict(alpha=0.5)):
        with pytest.raises(ValueError, match="delta"):
            serve.forward(stream, None, nw, w, up, down, t, **bad)


def test_training_step_of_layers_in_a_graph():
    """Two layers of linear, dropout within the join, and their backward by the operators' own calls, captured with the step's
    advance; each replay against the eager step of that number."""
    require_gpu()
    rnd = _rnd(9)
    rows, D, F = 96, 256, 520
    layers = [(rnd(F, D, dtype=BF, scale=0.06), rnd(F), rnd(D, F, dtype=BF, scale=0.05), (1 + rnd(D, scale=0.1)).to(BF),
               (1 + rnd(D, scale=0.1)).to(BF), rnd(D, dtype=BF)) for _ in range(2)]
    x0, dy = rnd(rows, D, dtype=BF), rnd(rows, D, dtype=BF)

    def step(rng):
        st, x, saved = x0, x0, []
        for k, (w1, b1, w2, nw, pw, gate) in enumerate(layers):
            pre = torch.empty(rows, F, dtype=BF, device="cuda")
            h = tw.linear(x, w1, bias=b1, act="silu", pre=pre)
            y = tw.linear(h, w2, dtype=F32)
            j = tw.join_rms_norm(st, y, nw, post_weight=pw, gate=gate, p=0.1, rng=rng, site=k, stats=True)
            saved.append((x, pre, h, y, j))
            st, x = j.residual, j.out
        grads, d_st, d_x = [st, x], None, dy
        for k in (1, 0):
            w1, b1, w2, nw, pw, gate = layers[k]
            xin, pre, h, y, j = saved[k]
            gj = tw.join_rms_norm_bwd(d_x, j.residual, j.rstd, y, nw, post_weight=pw, post_rstd=j.post_rstd, gate=gate, p=0.1, rng=rng,
                                      site=k, d_residual=d_st)
            g2 = tw.linear_bwd(gj.dy, h, w2, bias=False)
            g1 = tw.linear_bwd(g2.dx, xin, w1, act="silu", pre=pre)
            grads += [t for t in (*gj, *g2, *g1) if t is not None]
            d_st, d_x = gj.dr, g1.dx
        return grads

    rng = tw.make_rng(77, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(rng)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rng[1].add_(1)
        out = step(rng)
    for i in range(1, 5):
        graph.replay()
        want = step(tw.make_rng(77, i))
        torch.cuda.synchronize()
        assert len(out) == len(want)
        for a, b in zip(out, want):
            assert torch.equal(a, b)
