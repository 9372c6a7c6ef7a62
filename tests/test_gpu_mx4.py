"""MX4 on the GPU: quantisation bit for bit against the definition, the values back exactly, products against float64
within counted roundings (bit for bit where sums are exact), widths and sizes around every tile, special blocks, other
streams, graphs, and the FFN behind an MX4 gate."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw

import mx4_reference as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _guarded(shape, dtype):
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw[256:256 + n].view(dtype).view(shape), (raw[:256], raw[256 + n:])


def _check_guards(*guards):
    for before, behind in guards:
        assert bool((before == 0xA5).all()) and bool((behind == 0xA5).all()), "bytes outside an output were written"


def _rows(rng, rows, cols, dtype):
    """Rows over many scales, with values half way between two levels, zeros and signed zeros among them."""
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1)))
    ties = rng.random((rows, cols)) < 0.3
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 4.0])
    block = np.exp2(np.floor(np.log2(np.abs(v).max(1, keepdims=True))) - 2)
    v = np.where(ties, mids[rng.integers(0, len(mids), (rows, cols))] * block * rng.choice([-1, 1], (rows, cols)), v)
    v[rng.random((rows, cols)) < 0.05] = 0.0
    v[rng.random((rows, cols)) < 0.05] = -0.0
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


WIDTHS = [1, 7, 8, 31, 32, 33, 64, 100, 127, 128, 129, 500, 512, 513, 1000, 1990, 2048, 4096, 4104, 11008]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_quantize_and_back(cols, dtype):
    require_gpu()
    for rows in (1, 3, 37):
        print(f"[mx4] {rows}x{cols} {dtype}", flush=True)
        a = _rows(np.random.default_rng(cols + rows), rows, cols, dtype)
        qs, ss = tw.mx4_shapes(rows, cols)
        (q, g1), (s, g2) = _guarded(qs, torch.uint8), _guarded(ss, torch.uint8)
        tw.quantize_mx4(a.cuda(), out=(q, s))
        want_q, want_s = ref.pack(*ref.quantize(a.double().numpy()))
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)  # codes, and zeros behind the last column
        for dt in (BF, F32):
            back, g3 = _guarded((rows, cols), dt)
            tw.dequantize_mx4(q, s, cols, out=back)
            v = ref.values(want_q, want_s, cols)
            assert np.array_equal(back.cpu().double().numpy(), v)
            assert np.array_equal(np.signbit(back.cpu().double().numpy()), np.signbit(v))
            _check_guards(g3)
        _check_guards(g1, g2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_blocks(dtype):
    """Blocks of zeros, subnormals, the largest numbers, infinities and NaN: codes, and only their own block changes."""
    require_gpu()
    rng = np.random.default_rng(1)
    a = _rows(rng, 12, 160, F32).to(dtype).float()
    tiny = float(torch.finfo(F32).tiny)
    a[0, 32:64] = 0
    a[1, 32:64] *= 0
    a[1, 40] = float("nan")
    a[2, 33] = float("inf")
    a[3, 63] = -float("inf")
    a[4, :32] = a[4, :32].sign() * tiny / 64           # subnormal: the scale is held at 2^-127
    a[5, :32] = tiny * torch.arange(32)                # around the lowest scale
    a[6, 64:96] = a[6, 64:96].sign() * float(torch.finfo(dtype).max)
    a[7, 0] = float(torch.finfo(dtype).max)
    a[8, 5], a[8, 6] = float("nan"), float("inf")
    a = a.to(dtype)
    q, s = tw.quantize_mx4(a.cuda())
    want_q, want_s = ref.pack(*ref.quantize(a.double().numpy()))
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)
    assert want_s[1, 1] == want_s[2, 1] == want_s[3, 1] == want_s[8, 0] == 255 and want_s[0, 1] == 0
    back = tw.dequantize_mx4(q, s, 160, dtype=F32).cpu().double().numpy()
    v = ref.values(want_q, want_s, 160)
    assert np.array_equal(np.isnan(back), np.isnan(v)) and np.array_equal(back[~np.isnan(v)], v[~np.isnan(v)])


def _product_tol(xv, wv, y, dtype):
    """|y - y64|: at most one rounding of the absolute sum for every run of 8 products, every instruction, every wave
    and the final store."""
    size = np.abs(xv) @ np.abs(wv).T
    steps = xv.shape[1] / 8 + xv.shape[1] / 128 + 12
    tol = size * steps * U
    return tol + (0 if dtype == F32 else (np.abs(y) + tol) * 2.0 ** -8)


# rows and units below, at and above every tile's edge; widths with part blocks, part steps and part scale words
PRODUCTS = [(1, 1, 1), (1, 128, 16), (1, 4096, 1000), (2, 33, 17), (5, 520, 300), (15, 1990, 64), (16, 2048, 129),
            (17, 96, 31), (24, 2048, 250), (32, 1000, 48), (33, 640, 99), (63, 130, 100), (64, 512, 512), (65, 129, 65),
            (100, 1990, 130), (128, 256, 4), (200, 700, 511), (257, 4096, 300), (1003, 1990, 81),
            (65, 257, 128), (127, 300, 136), (128, 384, 128), (129, 385, 132), (130, 512, 192), (255, 640, 255)]


@pytest.mark.parametrize("n,cols,units", PRODUCTS)
def test_products(n, cols, units):
    require_gpu()
    rng = np.random.default_rng(n * 7 + cols + units)
    w = torch.from_numpy((rng.standard_normal((units, cols)) / np.sqrt(cols)).astype(np.float32))
    wq, ws = tw.quantize_mx4(w.cuda())
    wv = ref.values(*ref.pack(*ref.quantize(w.numpy())), cols)
    for xdt in (BF, F32):
        x = torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).to(xdt)
        if n > 3:
            x[3] = 0
        xv = ref.values(*ref.pack(*ref.quantize(x.double().numpy())), cols)
        y64 = xv @ wv.T
        for ydt in (BF, F32):
            print(f"[mx4 product] {n}x{cols}x{units} {xdt} {ydt}", flush=True)
            y, g = _guarded((n, units), ydt)
            tw.linear_mx4(x.cuda(), wq, ws, out=y)
            torch.cuda.synchronize()
            _check_guards(g)
            assert bool((np.abs(y.cpu().double().numpy() - y64) <= _product_tol(xv, wv, y64, ydt)).all())
            xq, xs = tw.quantize_mx4(x.cuda())
            z = tw.matmul_mx4(xq, xs, wq, ws, cols, dtype=ydt)
            assert bool((np.abs(z.cpu().double().numpy() - y64) <= _product_tol(xv, wv, y64, ydt)).all())
            again = tw.linear_mx4(x.cuda(), wq, ws, dtype=ydt)
            assert torch.equal(again, y)


@pytest.mark.parametrize("n,cols,units", [(4352, 640, 4352), (4099, 1990, 4611), (8192, 130, 2053), (8195, 384, 2304),
                                          (2304, 4096, 8192), (700, 2048, 5632), (1001, 1152, 1003), (90, 4096, 2056),
                                          (70, 4997, 2055), (127, 4100, 1500), (40003, 384, 130),
                                          (70, 600, 70003), (20, 1100, 132001)])
def test_large_products_are_exact(n, cols, units):
    """Small whole numbers: every sum is exact in fp32, whatever its order, so y is too. Covers whole grids of the
    tiled product with edges on both sides, against float64 on the GPU's own fp32-exact product."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    level = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0], device="cuda")
    sign = lambda *s: torch.randint(0, 2, s, generator=gen, device="cuda") * 2.0 - 1  # noqa: E731
    x = level[torch.randint(0, 6, (n, cols), generator=gen, device="cuda")] * sign(n, cols)
    w = level[torch.randint(0, 6, (units, cols), generator=gen, device="cuda")] * sign(units, cols)
    # a block's largest element decides its scale: make it 6 or 4, so that the elements are codes as they stand
    x[:, ::32], w[:, ::32] = 4, 6
    x *= torch.exp2(torch.randint(-3, 4, (n, 1), generator=gen, device="cuda").float())
    want = torch.matmul(x, w.t())  # whole multiples of one power of two a row, below 2^24 of it: exact
    wq, ws = tw.quantize_mx4(w)
    for xdt in (BF, F32):
        got = tw.linear_mx4(x.to(xdt), wq, ws, dtype=F32)
        assert torch.equal(got, want)
        assert torch.equal(tw.linear_mx4(x.to(xdt), wq, ws), want.to(BF))


@pytest.mark.parametrize("n,cols,units", [(100, 4096, 2048), (77, 3333, 4111), (300, 2050, 1024), (600, 1990, 1001),
                                          (130, 1100, 6000), (4400, 1000, 4352), (4107, 2999, 4333),
                                          # x quantised by the product, several tiles of tokens
                                          (24, 2048, 5632), (31, 1500, 3001), (60, 1500, 1500), (100, 1001, 2051), (200, 512, 1024),
                                          (300, 333, 700),
                                          # one stage of columns, whole and half, both tiles, edges, several tiles a workgroup
                                          (1500, 64, 1100), (2049, 128, 1003), (1300, 256, 1201), (131, 129, 12001),
                                          (4097, 200, 4352), (4100, 100, 4501), (9001, 31, 2055), (150, 255, 70001)])
def test_large_products(n, cols, units):
    """The tiles on ordinary values, against float64 of the values that the operands stand for."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(n, cols, generator=gen, device="cuda") * torch.exp(torch.randn(n, 1, generator=gen, device="cuda"))
    w = torch.randn(units, cols, generator=gen, device="cuda") / cols ** 0.5
    xq, xs = tw.quantize_mx4(x)
    wq, ws = tw.quantize_mx4(w)
    xv, wv = (tw.dequantize_mx4(*v, cols, dtype=F32).double() for v in ((xq, xs), (wq, ws)))
    want = torch.matmul(xv, wv.t())
    size = torch.matmul(xv.abs(), wv.abs().t())
    tol = size * ((cols / 8 + cols / 64 + 12) * U)
    y = tw.linear_mx4(x, wq, ws, dtype=F32)
    assert bool(((y.double() - want).abs() <= tol).all())
    y2 = tw.matmul_mx4(xq, xs, wq, ws, cols, dtype=F32)
    if tw.linear_mx4_ws(n, cols, units):  # the same product; one that quantises x adds in another order
        assert torch.equal(y2, y)
    assert bool(((y2.double() - want).abs() <= tol).all())
    b = tw.linear_mx4(x, wq, ws)
    assert torch.equal(b, y.to(BF))
    assert torch.equal(tw.linear_mx4(x, wq, ws), b)


@pytest.mark.parametrize("n,units", [(4, 40), (20, 40), (70, 70), (70, 300), (300, 200), (1500, 1100), (4500, 4500)])
@pytest.mark.parametrize("cols", [300, 100, 256])
def test_nan_blocks_mark_their_row_and_column(n, units, cols):
    require_gpu()
    rng = np.random.default_rng(n)
    x = torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.standard_normal((units, cols)).astype(np.float32)).cuda()
    clean = tw.linear_mx4(x, *tw.quantize_mx4(w), dtype=F32)
    x[2, cols - 10] = float("nan")
    w[7, 0] = float("inf")
    y = tw.linear_mx4(x, *tw.quantize_mx4(w), dtype=F32)
    bad = torch.zeros(n, units, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 7] = True, True
    assert bool((y.isnan() == bad).all()) and torch.equal(y[~bad], clean[~bad])


def test_empty():
    require_gpu()
    e = torch.empty(0, 300, device="cuda")
    q, s = tw.quantize_mx4(e)
    assert q.shape == (0, 192) and s.shape == (0, 16) and tw.dequantize_mx4(q, s, 300).shape == (0, 300)
    w = tw.quantize_mx4(torch.ones(5, 300, device="cuda"))
    assert tw.linear_mx4(e, *w).shape == (0, 5) and tw.matmul_mx4(q, s, *w, 300).shape == (0, 5)


@pytest.mark.parametrize("n", [3, 40, 100, 2100, 8200])
def test_other_stream_and_graph_replay(n):
    require_gpu()
    cols, units = 520, 2100
    x, w = torch.randn(n, cols, device="cuda"), torch.randn(units, cols, device="cuda")
    wq, ws = tw.quantize_mx4(w)
    want = tw.linear_mx4(x, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tw.linear_mx4(x, *tw.quantize_mx4(w))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    y, space = torch.empty(n, units, dtype=BF, device="cuda"), tw.alloc_workspace(tw.linear_mx4_ws(n, cols, units))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.linear_mx4(x, wq, ws, out=y, ws=space)
    for k in range(4):
        x.mul_(1.5).add_(0.1 * k)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tw.linear_mx4(x, wq, ws))
