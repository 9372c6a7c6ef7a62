"""The operators around the block as programs use them: a captured step that adds its own y, views that begin
anywhere, rows whose squares overflow a sum."""
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


@pytest.mark.parametrize("res", [F32, BF])
@pytest.mark.parametrize("cols", [16, 95, 200, 509, 512, 1000, 2050, 4096, 8200, 16383, 16384])
def test_norm_of_rows_whose_squares_overflow_a_sum(cols, res):
    """Elements far below the root of the largest number, whose squares add up to more than it: the norm, its codes
    and gradient are those of any other row. A mean of squares beyond fp32 still has rho = 0, and rows of ordinary
    size next to such ones keep their bits."""
    require_gpu()
    gen = torch.Generator().manual_seed(cols)
    rows = 19
    r = 1 + torch.rand(rows, cols, generator=gen)
    sizes = [1.0, 1e16, 1e17, 2e17, 5e17, 1e18, 3e18, 7e18, 8.5e18]  # rms up to 1.7e19
    for i in range(rows):
        r[i] *= sizes[i % len(sizes)]
    r[rows - 1] = 1e20  # its mean of squares is beyond fp32
    r = r.to(res)
    w = 1 + 0.3 * torch.randn(cols, generator=gen)
    got = tw.add_rms_norm(r.cuda(), w.cuda(), eps=EPS, out_dtype=F32, codes=True, rstd=True)
    x = r.double()[:-1]
    rho = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    # at most 32 squares a thread, 6 + 4 steps over lanes and 8 waves: 50 roundings of positive terms, which the root
    # halves; then mean (two), eps, root and quotient
    rel = (50 / 2 + 5) * 2.0 ** -24
    assert bool(((got.rstd.cpu().double()[:-1, None] - rho).abs() <= rho * rel).all())
    n = x * rho * w.double()
    assert bool(((got.out.cpu().double()[:-1] - n).abs() <= n.abs() * (rel + 2.0 ** -23)).all())
    q, s = tw.quantize_e4m3(got.out)
    assert torch.equal(q, got.codes) and torch.equal(s, got.scale)
    assert float(got.rstd[-1]) == 0 and bool((got.out[-1] == 0).all())
    plain = [i for i in range(rows) if i % len(sizes) == 0 and i < rows - 1]
    for a, b in zip(got, tw.add_rms_norm(r[plain].cuda(), w.cuda(), eps=EPS, out_dtype=F32, codes=True, rstd=True)):
        assert torch.equal(a[plain], b)
    g = torch.randn(rows, cols, generator=gen)
    dr, dw = tw.add_rms_norm_bwd(g[:-1].cuda(), r[:-1].cuda(), got.rstd[:-1].contiguous(), w.cuda())
    rs = got.rstd[:-1].cpu().double()[:, None]
    u, xh = g[:-1].double() * w.double(), x * rs
    size = rs * (u.abs() + xh.abs() * (u * xh).abs().mean(1, keepdim=True))
    want = rs * (u - xh * (u * xh).mean(1, keepdim=True))
    # the row's mean is off by at most 60 roundings of its absolute terms, the products by 6; then the type's own
    err, step = (dr.cpu().double() - want).abs(), torch.finfo(res).eps / 2
    assert bool((err <= size * (66 * 2.0 ** -24 + (step if res == BF else 0) * 1.01) + 2.0 ** -133).all())
