"""The residual-adding RMS norm on the GPU against float64: the stream bit for bit, the norm and both gradients within
bounds counted in roundings, the E4M3 codes against the row quantiser and against the fp32 norm, special rows,
buffers that are not asked for, the stream in place, other streams, graphs."""
from __future__ import annotations

import itertools

import pytest
import torch

from activation_sparse_ffn_03_amd import autograd as ag
from activation_sparse_ffn_03_amd import twell as tw

import norm_reference as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _rand(gen, *shape, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def _inputs(rows, cols, res, delta, w, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = _rand(gen, rows, cols, dtype=F32) * torch.exp(torch.randn(rows, 1, generator=gen))
    return r.to(res), None if delta is None else _rand(gen, rows, cols, scale=0.5, dtype=delta), \
        (1 + _rand(gen, cols, scale=0.3)).to(w)


def _guarded(shape, dtype):
    """A tensor inside a buffer filled with a byte pattern, and the buffer's bytes before and behind it."""
    n = torch.empty(0, dtype=dtype).element_size()
    for s in shape:
        n *= s
    raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw[256:256 + n].view(dtype).view(shape), (raw[:256], raw[256 + n:])


def _check_guards(*guards):
    for before, behind in guards:
        assert bool((before == 0xA5).all()) and bool((behind == 0xA5).all()), "bytes outside an output were written"


# widths: below and at one chunk, partial chunks, every register tile of the kernels and its borders, the widest
WIDTHS = [1, 7, 8, 9, 64, 511, 512, 513, 1000, 1024, 1999, 2048, 2056, 4095, 4096, 4104, 8192, 8200, 12345, 16384]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5])
def test_forward_widths(rows, cols):
    require_gpu()
    for k, (res, delta, out) in enumerate(itertools.product((BF, F32), (None, BF, F32), (BF, F32))):
        print(f"[norm] {rows}x{cols} {res} {delta} {out}", flush=True)
        _forward_case(rows, cols, res, delta, out, (BF, F32)[k % 2], seed=k)


@pytest.mark.parametrize("rows,cols", [(1024, 64), (1025, 513), (1030, 1000), (1027, 1999), (1024, 2048), (1026, 4096),
                                       (1031, 4090), (1024, 4104)])
@pytest.mark.parametrize("res,delta,out", [(BF, F32, BF), (F32, None, F32), (F32, BF, BF), (BF, BF, F32)])
def test_forward_many_rows(rows, cols, res, delta, out):
    """From 1024 rows on a wave takes a row; the last workgroup is not full."""
    require_gpu()
    _forward_case(rows, cols, res, delta, out, BF, seed=3)


def _forward_case(rows, cols, res, delta, out, wdt, seed):
    r, d, w = _inputs(rows, cols, res, delta, wdt, seed)
    if rows > 3:
        r[3] = 0
        if d is not None:
            d[3] = 0
    bufs, guards = zip(_guarded((rows, cols), res), _guarded((rows, cols), out), _guarded((rows, cols), torch.uint8),
                       _guarded((rows,), F32), _guarded((rows,), F32))
    got = tw.add_rms_norm(r.cuda(), w.cuda(), delta=None if d is None else d.cuda(), eps=EPS, out=bufs)
    torch.cuda.synchronize()
    _check_guards(*guards)
    want_r, n, rho = ref.forward64(r, d, w, EPS)
    assert torch.equal(got.residual.cpu(), want_r)
    o = got.out.cpu()
    assert bool(((o.double() - n).abs() <= ref.forward_tol(n, out)).all())
    assert bool(((got.rstd.cpu().double()[:, None] - rho).abs() <= rho * ((ref.ROW_ADDS + 1) / 2 + 4) * ref.U).all())
    # the codes: against the row quantiser on the fp32 norm, bit for bit
    n32 = o.cuda() if out == F32 else tw.add_rms_norm(
        r.cuda(), w.cuda(), delta=None if d is None else d.cuda(), eps=EPS,
        out=(None, torch.empty(rows, cols, device="cuda"), None, None, None)).out
    q, scale = tw.quantize_e4m3(n32)
    assert torch.equal(got.codes, q) and torch.equal(got.scale, scale)
    # and against the float64 norm
    s = got.scale.cpu().double()[:, None]
    v = ref.e4m3_values()[got.codes.cpu().long()]
    exact = n / s
    slack = ref.forward_tol(n, F32) / s + 4 * ref.U * exact.abs()
    assert bool(((v - exact).abs() <= ref.e4m3_tol(exact) + slack).all())
    top = n.abs().max(1, keepdim=True).values
    want_s = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert bool(((s - want_s).abs() <= want_s * ((ref.ROW_ADDS + 1) / 2 + 8) * ref.U).all())


def test_outputs_that_are_not_asked_for_and_the_stream_in_place():
    require_gpu()
    r, d, w = (v.cuda() for v in _inputs(37, 1030, BF, F32, BF))
    full = tw.add_rms_norm(r, w, delta=d, codes=True, rstd=True)
    for keep in itertools.product((False, True), repeat=4):
        if not any(keep):
            continue
        bufs = [torch.empty_like(full.residual) if keep[0] else None, torch.empty_like(full.out) if keep[1] else None,
                torch.empty_like(full.codes) if keep[2] else None, torch.empty_like(full.scale) if keep[2] else None,
                torch.empty_like(full.rstd) if keep[3] else None]
        got = tw.add_rms_norm(r, w, delta=d, out=bufs)
        for a, b in zip(got, full):
            assert a is None or torch.equal(a, b)
    stream = r.clone()
    got = tw.add_rms_norm(stream, w, delta=d, out=full._replace(residual=stream, out=torch.empty_like(full.out)))
    assert got.residual is stream and torch.equal(stream, full.residual) and torch.equal(got.out, full.out)


@pytest.mark.parametrize("cols", [1000, 4096])
@pytest.mark.parametrize("rows", [9, 1025])
def test_special_rows(rows, cols):
    """Zeros, NaN, infinities, an overflowing sum of squares, tiny and subnormal rows: as the definition has it, and
    no row touches another."""
    require_gpu()
    r, _, w = _inputs(rows, cols, F32, None, F32)
    plain = r.clone()
    r[0] = 0
    r[1, 5] = float("nan")
    r[2, 7] = float("inf")
    r[3] *= 1e30                    # squares overflow fp32: rho = 0
    r[4] = 1e-30 * plain[4]         # rho = 1 / sqrt(eps)
    r[5] = 1e-42 * plain[5].sign()  # subnormal
    r[6, 3] = -float("inf")
    w[11] = 0
    got = tw.add_rms_norm(r.cuda(), w.cuda(), codes=True, rstd=True)
    base = tw.add_rms_norm(plain.cuda(), w.cuda(), codes=True, rstd=True)
    torch.cuda.synchronize()
    out, codes, scale = got.out.cpu(), got.codes.cpu(), got.scale.cpu()
    assert bool((out[0] == 0).all()) and scale[0] == 1 and bool(((codes[0] & 127) == 0).all())
    assert bool(out[1].isnan().all()) and scale[1] == 1 and bool((codes[1] == 0x7F).all())
    for row, col in ((2, 7), (6, 3)):  # rho = 0: 0 everywhere and 0 * inf = NaN at the infinity
        assert bool(out[row, col].isnan()) and int(out[row].isnan().sum()) == 1 and scale[row] == 1
        assert codes[row, col] == 0x7F and int(((codes[row] & 127) != 0).sum()) == 1
    assert bool((out[3] == 0).all()) and scale[3] == 1
    for row in (4, 5):
        _, n, _ = ref.forward64(r[row:row + 1], None, w, EPS)
        # products below the normal range are held to 2^-149 steps each
        assert bool(((out[row:row + 1].double() - n).abs() <= ref.forward_tol(n, F32) + 2.0 ** -147).all())
    for a, b in zip(got, base):  # the rows without a special value
        assert torch.equal(a[7:], b[7:])
    q, s = tw.quantize_e4m3(got.out)
    assert torch.equal(q, got.codes) and torch.equal(s, got.scale)


def test_infinite_scale():
    """A weight that overflows the norm: scale inf, finite elements 0, infinities NaN, as the row quantiser has it."""
    require_gpu()
    r, _, w = _inputs(3, 520, F32, None, F32)
    w[9] = 3e38
    r[:, 9] = 4.0 * r.abs().max()
    got = tw.add_rms_norm(r.cuda(), w.cuda(), codes=True)
    q, s = tw.quantize_e4m3(got.out)
    assert bool(torch.isinf(got.scale).any())
    assert torch.equal(q, got.codes) and torch.equal(s, got.scale)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (5, 64), (4, 512), (130, 520), (131, 1000), (64, 1024),
                                       (2600, 1999), (2049, 2048), (33, 2056), (700, 4096), (515, 4099), (40, 8192),
                                       (9, 8200), (6, 16384), (7, 16383)])
def test_backward(rows, cols):
    require_gpu()
    for k, (res, grad, stream) in enumerate(itertools.product((BF, F32), (BF, F32), (True, False))):
        print(f"[norm bwd] {rows}x{cols} {res} {grad} {stream}", flush=True)
        r, _, w = _inputs(rows, cols, res, None, (BF, F32)[k % 2], seed=k)
        gen = torch.Generator().manual_seed(100 + k)
        g = _rand(gen, rows, cols, scale=0.1, dtype=grad)
        s = _rand(gen, rows, cols, scale=0.1, dtype=res) if stream else None
        if rows > 2:
            r[2] = 0
        rstd = tw.add_rms_norm(r.cuda(), w.cuda(), eps=EPS, rstd=True).rstd
        (dr, g1), (dw, g2) = _guarded((rows, cols), res), _guarded((cols,), F32)
        args = (g.cuda(), r.cuda(), rstd, w.cuda())
        tw.add_rms_norm_bwd(*args, d_residual=None if s is None else s.cuda(), out=(dr, dw))
        torch.cuda.synchronize()
        _check_guards(g1, g2)
        want_r, want_w = ref.backward64(g, s, r, rstd.cpu(), w)
        groups = tw.add_rms_norm_bwd_ws(rows, cols) // (4 * cols) or 1
        tol_r, tol_w = ref.backward_tol(g, s, r, rstd.cpu(), w, groups)
        assert bool(((dr.cpu().double() - want_r).abs() <= tol_r).all())
        assert bool(((dw.cpu().double() - want_w).abs() <= tol_w).all())
        again = tw.add_rms_norm_bwd(*args, d_residual=None if s is None else s.cuda())
        assert torch.equal(again[0], dr) and torch.equal(again[1], dw)  # a fixed order of sums


def test_backward_of_no_rows_is_zero():
    require_gpu()
    e = torch.empty(0, 72, device="cuda")
    dr, dw = tw.add_rms_norm_bwd(e, e, torch.empty(0, device="cuda"), torch.ones(72, device="cuda"))
    assert dr.shape == (0, 72) and bool((dw == 0).all())


def test_gradient_against_differences():
    """d/dt of sum(out * g) + sum(r' * s) along random directions, by central differences of the float64 definition."""
    require_gpu()
    rows, cols = 6, 264
    r, d, w = _inputs(rows, cols, F32, F32, F32, seed=5)
    gen = torch.Generator().manual_seed(9)
    g, s = _rand(gen, rows, cols), _rand(gen, rows, cols)

    def loss(r64, w64):
        rho = 1 / torch.sqrt((r64 * r64).mean(1, keepdim=True) + EPS)
        return (r64 * rho * w64 * g.double()).sum() + (r64 * s.double()).sum()

    got = tw.add_rms_norm(r.cuda(), w.cuda(), delta=d.cuda(), eps=EPS, rstd=True)
    dr, dw = tw.add_rms_norm_bwd(g.cuda(), got.residual, got.rstd, w.cuda(), d_residual=s.cuda())
    base = got.residual.cpu().double()
    h = 1e-6
    for seed in range(5):
        gen = torch.Generator().manual_seed(seed)
        vr, vw = torch.randn(rows, cols, generator=gen).double(), torch.randn(cols, generator=gen).double()
        slope = (loss(base + h * vr, w.double() + h * vw) - loss(base - h * vr, w.double() - h * vw)) / (2 * h)
        mine = (dr.cpu().double() * vr).sum() + (dw.cpu().double() * vw).sum()
        # differences are good to about h^2 and 1e-16 / h of the loss; the sums over 1848 fp32 values to their roundings
        size = (dr.cpu().double() * vr).abs().sum() + (dw.cpu().double() * vw).abs().sum()
        assert abs(float(slope - mine)) <= float(size) * 200 * ref.U + 1e-7 * abs(float(loss(base, w.double())))


@pytest.mark.parametrize("lead", [(7,), (2, 3)])
@pytest.mark.parametrize("with_delta", [True, False])
def test_autograd(lead, with_delta):
    """Gradients of every input through the autograd form, for a loss on both outputs, on each alone, and for an
    expanded gradient; a delta of another type gets its gradient in its own type."""
    require_gpu()
    cols = 136
    r, d, w = _inputs(6 if len(lead) == 2 else 7, cols, F32, BF, BF, seed=2)
    r, d = r.reshape(*lead, cols), d.reshape(*lead, cols)
    gen = torch.Generator().manual_seed(4)
    g, s = _rand(gen, *lead, cols), _rand(gen, *lead, cols)

    def leaves(dev, dt=None):
        return [v.to(dev, dt).requires_grad_() for v in ((r, d, w) if with_delta else (r, w))]

    def run(use, dev):
        v = leaves(dev, torch.float64 if dev == "cpu" else None)
        rr, dd, ww = v if with_delta else (v[0], None, v[1])
        if dev == "cpu":
            st = rr if dd is None else rr + dd
            out = st / torch.sqrt((st * st).mean(-1, keepdim=True) + EPS) * ww
        else:
            st, out = ag.add_rms_norm(rr, ww, dd, eps=EPS, out_dtype=F32)
        c = (lambda x: x.to(dev)) if dev != "cpu" else (lambda x: x.double())
        loss = {"both": lambda: (out * c(g)).sum() + (st * c(s)).sum(), "out": lambda: (out * c(g)).sum(),
                "stream": lambda: (st * c(s)).sum(), "expanded": lambda: out.sum() + st.sum()}[use]()
        loss.backward()
        return [x.grad for x in v]

    for use in ("both", "out", "stream", "expanded"):
        for got, want, leaf in zip(run(use, "cuda"), run(use, "cpu"), (r, d, w) if with_delta else (r, w)):
            if want is None or got is None:
                assert got is None and (want is None or not bool(want.any()))
                continue
            assert got.dtype == leaf.dtype and got.shape == leaf.shape
            # sums of up to cols terms in fp32, then the gradient's own rounding
            err = (got.cpu().double() - want).abs()
            assert bool((err <= ref.half_step(got.dtype) * want.abs() + 100 * ref.U * want.abs().max()).all()), use


def test_shared_weight_gradient_adds_up():
    require_gpu()
    w = torch.ones(64, device="cuda", requires_grad=True)
    x = torch.randn(5, 64, device="cuda")
    a = ag.add_rms_norm(x, w)[1]
    b = ag.add_rms_norm(2 * x + 1, w)[1]
    (a.sum() + b.sum()).backward()
    want = (a.detach() + b.detach()).double().sum(0)
    assert bool(((w.grad.double() - want).abs() <= 40 * ref.U * (a.detach().abs() + b.detach().abs()).sum(0)).all())


def test_other_stream_and_graph_replay():
    require_gpu()
    r, d, w = (v.cuda() for v in _inputs(70, 1100, BF, F32, BF))
    g = torch.randn(70, 1100, device="cuda")
    want = tw.add_rms_norm(r, w, delta=d, codes=True, rstd=True)
    want_b = tw.add_rms_norm_bwd(g, want.residual, want.rstd, w, d_residual=want.out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tw.add_rms_norm(r, w, delta=d, codes=True, rstd=True)
        got_b = tw.add_rms_norm_bwd(g, got.residual, got.rstd, w, d_residual=got.out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip([*got, *got_b], [*want, *want_b]):
        assert torch.equal(a, b)
    bufs = tw.alloc_norm(r, codes=True, rstd=True)
    grads = (torch.empty_like(r), torch.empty(1100, device="cuda"))
    ws = tw.alloc_workspace(tw.add_rms_norm_bwd_ws(70, 1100))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tw.add_rms_norm(r, w, delta=d, out=bufs)
        tw.add_rms_norm_bwd(g, bufs.residual, bufs.rstd, w, d_residual=bufs.out, out=grads, ws=ws)
    for k in range(4):
        r.add_(0.25 * k)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = tw.add_rms_norm(r, w, delta=d, codes=True, rstd=True)
        want_b = tw.add_rms_norm_bwd(g, want.residual, want.rstd, w, d_residual=want.out)
        for a, b in zip([*bufs, *grads], [*want, *want_b]):
            assert torch.equal(a, b)


def test_block_trains():
    """TwellBlock against the same block in float64 autograd, small enough that every gate unit stays packed."""
    require_gpu()
    torch.manual_seed(0)
    N, D, F = 48, 128, 256
    blk = ag.TwellBlock(D, F, cfg=ag.TwellConfig(tile_n=32, slots=32, row_cap=256, dense_frac=1.0), dtype=F32)
    with torch.no_grad():
        blk.norm.weight.mul_(1 + 0.2 * torch.randn(D, device="cuda"))
    r = torch.randn(N, D, device="cuda", requires_grad=True)
    d = torch.randn(N, D, device="cuda", requires_grad=True)
    t = torch.full((N,), 0.5, device="cuda")
    gy, gs = torch.randn(N, D, device="cuda"), torch.randn(N, D, device="cuda")
    st, y = blk(r, d, t)
    ((y * gy).sum() + (st * gs).sum()).backward()
    p64 = [v.detach().cpu().double().requires_grad_() for v in
           (r, d, blk.norm.weight, blk.ffn.w_gate_t, blk.ffn.w_up_t, blk.ffn.w_down)]
    s64 = p64[0] + p64[1]
    x = s64 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-6) * p64[2]
    h = torch.relu(x @ p64[3].T - 0.5)
    y64 = (h * (x @ p64[4].T)) @ p64[5]
    ((y64 * gy.cpu().double()).sum() + (s64 * gs.cpu().double()).sum()).backward()
    assert float((y.detach().cpu().double() - y64).abs().max()) <= 1e-4 * float(y64.detach().abs().max())
    for a, b in zip((r, d, blk.norm.weight, blk.ffn.w_gate_t, blk.ffn.w_up_t, blk.ffn.w_down), p64):
        # fp32 sums of at most a few hundred terms of mixed sign
        assert float((a.grad.cpu().double() - b.grad).abs().max()) <= 1e-4 * float(b.grad.abs().max())


def test_more_rows_than_a_launch_takes():
    """Rows behind the first launch's 2^22 come out as they do alone."""
    require_gpu()
    rows, cols = 2 * (1 << 22) + 5, 9
    g = torch.Generator(device="cuda").manual_seed(5)
    r = torch.randn(rows, cols, generator=g, device="cuda").to(BF)
    d = torch.randn(rows, cols, generator=g, device="cuda")
    w = torch.randn(cols, generator=g, device="cuda")
    got = tw.add_rms_norm(r, w, delta=d, eps=EPS, codes=True, rstd=True)
    for at in (0, (1 << 22) - 3, (1 << 23) - 3, rows - 5):
        part = slice(at, at + 7)
        want = tw.add_rms_norm(r[part].clone(), w, delta=d[part].clone(), eps=EPS, codes=True, rstd=True)
        for a, b in zip(got, want):
            assert torch.equal(a[part], b)
