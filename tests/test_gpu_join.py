"""The join of a block's output to the stream and dropout on the GPU: masks bit for bit against the generator in whole
numbers, the stream, norm and gradients against float64 within bounds counted in roundings, special rows, buffers that are
not asked for, the stream in place, other streams, graphs that advance the generator."""
from __future__ import annotations

import itertools

import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw

import join_reference as jr
import norm_reference as ref
from gpu_util import require_gpu
from test_gpu_norm import _check_guards, _guarded, _rand

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
SEED, STEP, SITE = (0x9E21 << 40) + 77, (1 << 32) + 3, 9


def _rng():
    return tw.make_rng(SEED, STEP)


# ---------------------------------------------------------------- dropout

# below, at and above a generator block, partial blocks, every width of a workgroup and its borders
WIDTHS = [1, 5, 7, 8, 9, 63, 64, 65, 256, 257, 999, 1024, 1030, 2048, 2049, 5000]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_mask_and_values(cols, dtype):
    require_gpu()
    for rows, p in ((1, 0.1), (37, 0.5), (300, 0.03)):
        x = _rand(torch.Generator().manual_seed(rows), rows, cols, dtype=dtype)
        out, guard = _guarded((rows, cols), dtype)
        tw.dropout(x.cuda(), _rng(), p, site=SITE, out=out)
        torch.cuda.synchronize()
        _check_guards(guard)
        keep = jr.kept(rows, cols, p, SEED, STEP, SITE)
        want = torch.where(keep, x.float() * jr.factor(p), torch.zeros(())).to(dtype)  # one product, one rounding
        assert torch.equal(out.cpu(), want)
        inplace = x.cuda()
        assert tw.dropout(inplace, _rng(), p, site=SITE, out=inplace) is inplace and torch.equal(inplace, out)


def test_mask_depends_on_each_of_its_inputs():
    require_gpu()
    x = torch.ones(64, 512, device="cuda")
    masks = [tw.dropout(x, tw.make_rng(s, t), 0.5, site=i) > 0 for s, t, i in
             ((1, 0, 0), (2, 0, 0), (1 + (1 << 40), 0, 0), (1, 1, 0), (1, 0, 1), (-1, 0, 0))]
    for a, b in itertools.combinations(masks, 2):
        share = float((a != b).float().mean())
        assert 0.4 < share < 0.6  # 32768 fair coins: 36 standard deviations
    assert torch.equal(masks[0], tw.dropout(x, tw.make_rng(1, 1 << 32), 0.5) > 0)  # the step counts modulo 2^32
    assert torch.equal(masks[5].cpu(), jr.kept(64, 512, 0.5, -1, 0, 0))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -16, 0.25, 1 - 2.0 ** -16, 1.0])
def test_shares(p):
    """The kept share is the one that the factor stands for; p 0 keeps all bits, p 1 keeps nothing; what is dropped is 0
    whatever it holds."""
    require_gpu()
    n = 1 << 20
    x = torch.full((n // 1024, 1024), float("nan"), device="cuda")
    got = tw.dropout(x, _rng(), p, site=SITE)
    share = float((got == 0).float().mean())
    want = jr.threshold(p) / 65536
    assert abs(share - want) <= 6 * (want * (1 - want) / n) ** 0.5  # six standard deviations
    assert bool(((got == 0) | got.isnan()).all())
    y = _rand(torch.Generator().manual_seed(1), 8, 1024).cuda()
    got = tw.dropout(y, _rng(), p)
    if jr.threshold(p) == 0:
        assert torch.equal(got, y)
    if p == 1:
        assert torch.equal(got, torch.zeros_like(y))


def test_many_short_rows():
    """More rows than one launch holds; rows' numbers go on."""
    require_gpu()
    rows = (1 << 29) + 70
    x = torch.ones(rows, 1, dtype=BF, device="cuda")
    got = tw.dropout(x, _rng(), 0.5, site=SITE, out=x)
    for first in (0, (1 << 29) - 40, rows - 40):
        keep = jr.kept(40, 1, 0.5, SEED, STEP, SITE, first)
        assert torch.equal(got[first:first + 40].cpu() > 0, keep)


# ---------------------------------------------------------------- join

def _inputs(rows, cols, res, y, w, post, gates, seed):
    gen = torch.Generator().manual_seed(seed)
    r = (_rand(gen, rows, cols) * torch.exp(torch.randn(rows, 1, generator=gen))).to(res)
    b = (_rand(gen, rows, cols, scale=0.5) * torch.exp(torch.randn(rows, 1, generator=gen))).to(y)
    wt = (1 + _rand(gen, cols, scale=0.3)).to(w)
    pw = (0.7 + _rand(gen, cols, scale=0.3)).to(w) if post else None
    gate = None
    if gates:
        gate = (0.5 + _rand(gen, gates, cols, scale=0.4)).to(w)
        gate = gate[0] if gates == 1 and seed % 2 else gate
    if rows > 3:
        r[3] = 0
        b[3] = 0
    return r, b, wt, pw, gate


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _forward(rows, cols, res, y, w, post, gates, alpha, p, out_t, seed):
    r, b, wt, pw, gate = _inputs(rows, cols, res, y, w, post, gates, seed)
    print(f"[join] {rows}x{cols} {res} {y} {w} post={post} gates={gates} alpha={alpha} p={p} {out_t}", flush=True)
    bufs, guards = zip(_guarded((rows, cols), res), _guarded((rows, cols), out_t), _guarded((rows, cols), torch.uint8),
                       _guarded((rows,), F32), _guarded((rows,), F32), _guarded((rows,), F32))
    bufs = list(bufs)
    if not post:
        bufs[5] = None
    rg, bg, wg, pg, gg = _cuda(r, b, wt, pw, gate)
    got = tw.join_rms_norm(rg, bg, wg, post_weight=pg, gate=gg, alpha=alpha, eps=EPS, p=p, rng=_rng() if p else None,
                           site=SITE, out=bufs)
    torch.cuda.synchronize()
    _check_guards(*guards)
    keep = jr.kept(rows, cols, p, SEED, STEP, SITE) if p else None
    want, rho_y = jr.stream64(r, b, pw, gate, alpha, EPS, keep, p)
    st = got.residual.cpu()
    assert bool(((st.double() - want).abs() <= jr.stream_tol(r, b, pw, gate, alpha, EPS, keep, p)).all())
    rel = (ref.ROW_ADDS + 1) / 2 + 4
    if post:
        assert bool(((got.post_rstd.cpu().double()[:, None] - rho_y).abs() <= rho_y * rel * ref.U).all())
    # the norm is that of the stream as stored, with add_rms_norm's arithmetic
    same = tw.add_rms_norm(got.residual, wg, eps=EPS, out_dtype=out_t, codes=True, rstd=True)
    assert torch.equal(got.out, same.out) and torch.equal(got.codes, same.codes)
    assert torch.equal(got.scale, same.scale) and torch.equal(got.rstd, same.rstd)
    return (r, b, wt, pw, gate), keep, got


# every thread layout of the kernels and its borders
JOIN_WIDTHS = [1, 7, 8, 9, 128, 129, 250, 256, 512, 513, 1000, 1024, 1999, 2048, 2056, 4096, 4097, 8192, 8200, 12345, 16384]


@pytest.mark.parametrize("cols", JOIN_WIDTHS)
def test_forward_widths(cols):
    require_gpu()
    k = 0
    for res, y in itertools.product((BF, F32), repeat=2):
        for post, gates, alpha, p in ((True, 1, 1.0, 0.0), (True, 3, 0.7, 0.2), (False, 6, 1.0, 0.1), (True, 0, 1.5, 0.5), (False, 0, 1.0, 0.0)):
            _forward(6, cols, res, y, (BF, F32)[k % 2], post, gates, alpha, p, (BF, F32)[k // 2 % 2], seed=k)
            k += 1


@pytest.mark.parametrize("rows,cols", [(1, 4096), (1025, 95), (700, 1999), (515, 2048), (130, 8200)])
def test_forward_rows(rows, cols):
    require_gpu()
    for k, gates in enumerate((0, 1, rows, 5)):
        if gates == 0 or rows % gates == 0:
            _forward(rows, cols, BF, F32, BF, True, gates, 1.0, 0.1, BF, seed=k)


@pytest.mark.parametrize("cols", [5, 95, 1000, 4096, 8200])
def test_without_options_it_is_add_rms_norm(cols):
    require_gpu()
    for res, y in itertools.product((BF, F32), repeat=2):
        r, b, w, _, _ = _cuda(*_inputs(33, cols, res, y, BF, False, 0, 1))
        a = tw.join_rms_norm(r, b, w, eps=EPS, codes=True, stats=True)
        c = tw.add_rms_norm(r, w, delta=b, eps=EPS, codes=True, rstd=True)
        assert a.post_rstd is None
        for x, z in zip(a, c):
            assert torch.equal(x, z)


@pytest.mark.parametrize("cols", [7, 250, 1999, 4096])
def test_dropout_within_is_dropout_before(cols):
    """The mask is the one that dropout makes of the same rows, and what is dropped does not reach the stream."""
    require_gpu()
    r, b, w, _, _ = _cuda(*_inputs(65, cols, F32, F32, F32, False, 0, 2))
    b = torch.where(tw.dropout(torch.ones_like(b), _rng(), 0.3, site=SITE) > 0, b, float("inf"))
    one = tw.join_rms_norm(r, b, w, p=0.3, rng=_rng(), site=SITE)
    two = tw.join_rms_norm(r, tw.dropout(b, _rng(), 0.3, site=SITE), w)
    assert bool(one.residual.isfinite().all())
    assert torch.equal(one.residual, two.residual) and torch.equal(one.out, two.out)


def test_outputs_that_are_not_asked_for_and_the_stream_in_place():
    require_gpu()
    r, b, w, pw, gate = _cuda(*_inputs(36, 1030, BF, F32, BF, True, 4, 0))
    kw = dict(post_weight=pw, gate=gate, alpha=0.9, p=0.2, rng=_rng(), site=SITE)
    full = tw.join_rms_norm(r, b, w, codes=True, stats=True, **kw)
    for keep in itertools.product((False, True), repeat=5):
        if not any(keep):
            continue
        keep = keep[:3] + keep[2:]
        bufs = [torch.empty_like(f) if k else None for f, k in zip(full, keep)]
        for a, c in zip(tw.join_rms_norm(r, b, w, out=bufs, **kw), full):
            assert a is None or torch.equal(a, c)
    stream = r.clone()
    got = tw.join_rms_norm(stream, b, w, out=full._replace(residual=stream, out=torch.empty_like(full.out)), **kw)
    assert got.residual is stream and torch.equal(stream, full.residual) and torch.equal(got.out, full.out)


def test_special_rows():
    """Zeros, rows whose squares overflow fp32's sum, infinity and NaN: other rows are as they are alone."""
    require_gpu()
    cols = 515
    r, b, w, pw, gate = _inputs(8, cols, F32, F32, F32, True, 1, 3)
    b[0] = 0
    b[1] *= 1e18
    b[2, 7] = float("inf")
    b[4, 9] = float("nan")
    b[5] *= 1e-30
    r[6] = 0
    rg, bg, wg, pg, gg = _cuda(r, b, w, pw, gate)
    got = tw.join_rms_norm(rg, bg, wg, post_weight=pg, gate=gg, stats=True, codes=True)
    for i in range(8):
        alone = tw.join_rms_norm(rg[i:i + 1].clone(), bg[i:i + 1].clone(), wg, post_weight=pg, gate=gg, stats=True, codes=True)
        for a, c in zip(got, alone):
            assert torch.equal(a[i:i + 1].view(torch.uint8) if a.dtype == torch.uint8 else a[i:i + 1].nan_to_num(7.0), c if c.dtype == torch.uint8 else c.nan_to_num(7.0))
    ok = [0, 1, 3, 5, 6, 7]
    want, rho_y = jr.stream64(r[ok], b[ok], pw, gate, 1.0, EPS, None, 0)
    tol = jr.stream_tol(r[ok], b[ok], pw, gate, 1.0, EPS, None, 0)
    assert bool(((got.residual[ok].cpu().double() - want).abs() <= tol).all())
    assert bool(got.residual[4].isnan().all()) and bool(got.residual[2, 7].isnan())
    assert torch.equal(got.residual[2, :7], rg[2, :7])  # the row's rho_y is 0


def test_more_rows_than_a_launch_holds():
    require_gpu()
    rows, cols = (1 << 22) + 37, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = torch.randn(rows, cols, generator=gen, device="cuda")
    y = torch.randn(rows, cols, generator=gen, device="cuda")
    gate = torch.randn(rows, cols, generator=gen, device="cuda")
    w = torch.ones(cols, device="cuda")
    got = tw.join_rms_norm(r, y, w, gate=gate, p=0.5, rng=_rng(), site=SITE).residual
    want = r + gate * tw.dropout(y, _rng(), 0.5, site=SITE)
    # the kernel adds the product unrounded: one rounding of the product apart
    assert bool(((got - want).abs() <= (want.abs() + (gate * y * 2).abs()) * 2.0 ** -22).all())
    keep = jr.kept(30, cols, 0.5, SEED, STEP, SITE, (1 << 22) - 10)
    part = slice((1 << 22) - 10, (1 << 22) + 20)
    assert torch.equal((got[part] == r[part]).cpu(), ~keep)


# ---------------------------------------------------------------- gradients

def _backward(rows, cols, res, y, g_t, w, post, gates, alpha, p, stream, seed):
    print(f"[join_bwd] {rows}x{cols} {res} {y} {g_t} post={post} gates={gates} alpha={alpha} p={p} stream={stream}", flush=True)
    r, b, wt, pw, gate = _inputs(rows, cols, res, y, w, post, gates, seed)
    gen = torch.Generator().manual_seed(seed + 1000)
    g = _rand(gen, rows, cols, scale=0.1, dtype=g_t)
    s = _rand(gen, rows, cols, scale=0.1, dtype=res) if stream else None
    rho = (1 / torch.sqrt((r.double() ** 2).mean(1) + EPS)).float()
    rho_y = (1 / torch.sqrt((b.double() ** 2).mean(1) + EPS)).float() if post else None
    bufs, guards = zip(_guarded((rows, cols), res), _guarded((rows, cols), y), _guarded((cols,), F32),
                       _guarded((cols,), F32), _guarded((1,) if gate is None else tuple(gate.shape), F32))
    bufs = [bufs[0], bufs[1], bufs[2], bufs[3] if post else None, None if gate is None else bufs[4]]
    need = tw.join_rms_norm_bwd_ws(rows, cols, post, 0 if gate is None else gates)
    ws, ws_guard = _guarded((max(need, 16),), torch.uint8)
    rg, bg, wg, pg, gg, dg, sg, rh, ry = _cuda(r, b, wt, pw, gate, g, s, rho, rho_y)
    kw = dict(post_weight=pg, post_rstd=ry, gate=gg, alpha=alpha, p=p, rng=_rng() if p else None, site=SITE, d_residual=sg)
    got = tw.join_rms_norm_bwd(dg, rg, rh, bg, wg, out=bufs, ws=ws, **kw)
    torch.cuda.synchronize()
    _check_guards(*guards, ws_guard)
    keep = jr.kept(rows, cols, p, SEED, STEP, SITE) if p else None
    args = (g, s, r, rho, b, rho_y, wt, pw, gate, alpha, keep, p)
    for name, a, want, tol in zip(got._fields, got, jr.backward64(*args), jr.backward_tol(*args)):
        assert (a is None) == (want is None), name
        if a is not None:
            err = (a.cpu().double().reshape(want.shape) - want).abs()
            assert bool((err <= tol).all()), (name, float((err / tol.clamp(min=1e-300)).max()))
    again = tw.join_rms_norm_bwd(dg, rg, rh, bg, wg, **kw)
    for a, c in zip(got, again):  # the same bits every time
        assert a is None or torch.equal(a, c)


@pytest.mark.parametrize("cols", JOIN_WIDTHS)
def test_backward_widths(cols):
    require_gpu()
    k = 0
    for res, y in itertools.product((BF, F32), repeat=2):
        for post, gates, alpha, p, stream in ((True, 1, 1.0, 0.1, True), (True, 7, 0.7, 0.0, False), (False, 35, 1.0, 0.1, True),
                                              (False, 0, 1.0, 0.3, False), (True, 5, 1.0, 0.5, True)):
            _backward(35, cols, res, y, (BF, F32)[k % 2], (F32, BF)[k // 2 % 2], post, gates, alpha, p, stream, seed=k)
            k += 1


@pytest.mark.parametrize("rows,cols", [(1, 64), (1, 2048), (2, 100), (1000, 95), (1300, 250), (2040, 500), (1200, 1000), (900, 2048),
                                       (520, 4096), (300, 8192), (260, 16384)])
def test_backward_rows(rows, cols):
    """One workgroup and many; gates that are one, as many as rows, shared by parts of a workgroup's rows and by several
    workgroups, more of them than workgroups."""
    require_gpu()
    for k, gates in enumerate((0, 1, rows, rows // 2, 4, rows // 260 and rows // (rows // 260), 10)):
        if gates == 0 or rows % gates == 0:
            _backward(rows, cols, BF, F32, BF, F32, True, gates, 1.0, 0.1, k % 2 == 0, seed=k)


@pytest.mark.parametrize("gates", [0, 1, 6])
def test_no_rows(gates):
    require_gpu()
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    w, gate = torch.ones(96, device="cuda"), e(gates, 96) if gates else None
    got = tw.join_rms_norm(e(0, 96), e(0, 96), w, post_weight=w, gate=gate)
    assert got.out.shape == (0, 96)
    out = [e(0, 96), e(0, 96)] + [torch.full(s, 5.0, device="cuda") for s in ((96,), (96,))] + [None if gate is None else torch.full((gates, 96), 5.0, device="cuda")]
    grads = tw.join_rms_norm_bwd(e(0, 96), e(0, 96), e(0), e(0, 96), w, post_weight=w, post_rstd=e(0), gate=gate, out=out)
    for g in grads[2:]:
        assert g is None or bool((g == 0).all())
    assert tw.dropout(e(0, 96), _rng(), 0.5).shape == (0, 96)


def test_dropped_infinities_leave_the_gradient_finite():
    require_gpu()
    rows, cols = 40, 300
    r, b, w, _, gate = _cuda(*_inputs(rows, cols, F32, F32, F32, False, 1, 5))
    keep = tw.dropout(torch.ones_like(b), _rng(), 0.4, site=SITE) > 0
    b = torch.where(keep, b, float("nan"))
    f = tw.join_rms_norm(r, b, w, gate=gate, p=0.4, rng=_rng(), site=SITE, stats=True)
    g = tw.join_rms_norm_bwd(torch.ones_like(r), f.residual, f.rstd, b, w, gate=gate, p=0.4, rng=_rng(), site=SITE)
    assert all(bool(t.isfinite().all()) for t in g if t is not None)
    assert bool((g.dy[~keep] == 0).all())


# ---------------------------------------------------------------- streams and graphs

def test_other_stream_and_graph_with_an_advancing_generator():
    """A captured forward and backward; the step is advanced within the graph, eager work and other replays lie between."""
    require_gpu()
    rows, cols = 300, 1000
    r, b, w, pw, gate = _cuda(*_inputs(rows, cols, BF, F32, BF, True, 3, 4))
    g = torch.randn(rows, cols, device="cuda")

    def step(rng):
        f = tw.join_rms_norm(r, b, w, post_weight=pw, gate=gate, p=0.2, rng=rng, site=1, stats=True)
        d = tw.dropout(f.out, rng, 0.3, site=2)
        return [*f, d, *tw.join_rms_norm_bwd(g, f.residual, f.rstd, b, w, post_weight=pw, post_rstd=f.post_rstd, gate=gate, p=0.2,
                                             rng=rng, site=1, d_residual=f.residual)]

    rngs, graphs, outs = [tw.make_rng(5, 10), tw.make_rng(6, 20)], [], []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for rng in rngs:
            step(rng)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for rng in rngs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rng[1].add_(1)
            outs.append(step(rng))
        graphs.append(graph)
    for i in range(1, 5):
        for (seed, first), graph, out in zip(((5, 10), (6, 20)), graphs, outs):
            graph.replay()
            want = step(tw.make_rng(seed, first + i))
            torch.cuda.synchronize()
            for a, c in zip(out, want):
                assert a is None or torch.equal(a, c)
