"""The operators around the block as programs use them: a captured step that adds its own y, views that begin
anywhere."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_ffn_03_amd import autograd as ag
from activation_sparse_ffn_03_amd import twell as tw
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.mark.parametrize("gate", ["bf16", "fp8", "mx4"])
def test_capture_keeps_the_pending_delta(gate):
    """y is the delta of the next call: recording that call neither uses y up nor changes it, and every replay adds the
    y of the one before, as a chain of eager calls does."""
    require_gpu()
    N, D, F = 4, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dims = tw.make_dims(N, D, F, 64, 64, 0, 8, 0)
    w = (rnd(F, D) / D ** 0.5).to(BF)
    w = {"bf16": lambda: w, "fp8": lambda: tw.quantize_e4m3(w), "mx4": lambda: tw.quantize_mx4(w)}[gate]()
    weights = ((1 + 0.2 * rnd(D)).to(BF), w, (rnd(F, D) / D ** 0.5).to(BF), (rnd(F, D) / F ** 0.5).to(BF),
               torch.full((N,), 1.15, device="cuda"))
    stream, delta = rnd(N, D).to(BF), rnd(N, D)
    want_stream = stream.clone()
    serve, eager = tw.TwellServe(dims, gate, EPS), tw.TwellServe(dims, gate, EPS)
    y, want = serve.forward(stream, delta, *weights), eager.forward(want_stream, delta, *weights)
    graph = serve.capture(stream, y, *weights)
    torch.cuda.synchronize()
    assert torch.equal(stream, want_stream) and torch.equal(y, want)  # nothing has run yet
    for _ in range(4):
        graph.replay()
        want = eager.forward(want_stream, want, *weights)
        torch.cuda.synchronize()
        assert torch.equal(stream, want_stream) and torch.equal(y, want)


def _norm64(r, w):
    x = r.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cols", [1999, 1000, 5])
def test_autograd_takes_views_that_begin_anywhere(cols, dtype):
    """Slices of rows of an odd width, views into a flat buffer (of the weight, too), and the gradient that cat hands
    to its second input: none begins at 16 bytes, values and gradients are those of the same rows alone."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    rows = 5

    def view(*shape):  # an element behind an aligned address
        n = 1
        for s in shape:
            n *= s
        return rnd(n + 1)[1:].view(shape)

    r, d, w, top = view(rows, cols), rnd(rows + 1, cols)[1:], view(cols), rnd(1, cols)
    assert any(t.data_ptr() % 16 for t in (r, d, w))

    def run(make):
        v = [make(t) for t in (r, d, w, top)]
        for t in v:
            t.requires_grad_()
        st, out = ag.add_rms_norm(v[0], v[2], v[1], eps=EPS)
        both = torch.cat([v[3], out]) * torch.cat([st, v[3]])
        both.float().square().sum().backward()
        return [st, out] + [t.grad for t in v]

    for got, want in zip(run(lambda t: t.detach()), run(lambda t: t.detach().clone())):
        assert torch.equal(got, want)
    st, out = ag.add_rms_norm(r.detach(), w.detach(), d.detach(), eps=EPS)
    assert torch.equal(st, (r.detach().float() + d.detach().float()).to(dtype))
    n = _norm64(st, w.detach())
    # the row's sum of squares: at most cols / 2 + 8 roundings of fp32 reach the norm, then its own
    assert bool(((out.double() - n).abs() <= n.abs() * ((cols / 2 + 8) * 2.0 ** -24 + torch.finfo(dtype).eps / 2 * 1.01)).all())
    alone = ag.add_rms_norm(r.detach(), w.detach(), eps=EPS)
    assert alone[0].data_ptr() == r.data_ptr()  # nothing to add: the stream itself
    assert torch.equal(alone[1], ag.add_rms_norm(r.detach().clone(), w.detach().clone(), eps=EPS)[1])
