"""The operators around the block at sizes that take kernel variants of their own (fewer tokens than a tile in whole
stages, direct tiles of 64, one half stage of columns, narrow and wide rows of any width), and products over the whole
range of scales."""
from __future__ import annotations

import pytest
import torch

import test_gpu_norm as norm
from activation_sparse_ffn_03_amd import twell as tw
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

EXACT = [(64, 4096, 11008), (100, 2048, 12001), (17, 4096, 11008), (20000, 512, 96), (100001, 1000, 65), (16384, 4096, 100),
         (140, 100, 30001), (200, 128, 20000)]


def _whole(gen, n, cols, first):
    """Small whole numbers that are codes as they stand: `first` at every block's head makes its scale a power of two."""
    level = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0, -1.0, -2.0, -3.0, -4.0, -6.0], device="cuda")
    v = level[torch.randint(0, len(level), (n, cols), generator=gen, device="cuda")]
    v[:, ::32] = first
    return v


@pytest.mark.parametrize("n,cols,units", EXACT)
def test_products_are_exact(n, cols, units):
    """Every sum of whole numbers below 2^24 is exact in fp32, whatever its order, so y is too: the product that
    quantises x and the one of quantised rows, against float64."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, w = _whole(gen, n, cols, 4), _whole(gen, units, cols, 6)
    assert 36 * cols < 1 << 24
    x *= torch.exp2(torch.randint(-3, 4, (n, 1), generator=gen, device="cuda").float())
    want = torch.matmul(x.double(), w.double().t().contiguous()).float()
    wq, ws = tw.quantize_mx4(w)
    for xdt in (BF, F32):
        print(f"[exact] {n}x{cols}x{units} {xdt}", flush=True)
        assert torch.equal(tw.linear_mx4(x.to(xdt), wq, ws, dtype=F32), want)
        assert torch.equal(tw.linear_mx4(x.to(xdt), wq, ws), want.to(BF))
    xq, xs = tw.quantize_mx4(x)
    assert torch.equal(tw.matmul_mx4(xq, xs, wq, ws, cols, dtype=F32), want)
    assert torch.equal(tw.matmul_mx4(xq, xs, wq, ws, cols), want.to(BF))


NAN = [(100, 4096, 2048), (64, 2000, 12001)]


@pytest.mark.parametrize("n,cols,units", NAN)
def test_nan_blocks_mark_their_row_and_column(n, cols, units):
    """Fewer tokens than a tile."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, w = (torch.randn(r, cols, generator=gen, device="cuda") for r in (n, units))
    clean = tw.linear_mx4(x, *tw.quantize_mx4(w), dtype=F32)
    x[2, cols - 10], x[n - 1, 0] = float("nan"), float("-inf")
    w[7, 0], w[units - 1, cols - 1] = float("inf"), float("nan")
    y = tw.linear_mx4(x, *tw.quantize_mx4(w), dtype=F32)
    bad = torch.zeros(n, units, dtype=torch.bool, device="cuda")
    for i, c in ((2, 7), (n - 1, units - 1)):
        bad[i], bad[:, c] = True, True
    assert bool((y.isnan() == bad).all()) and torch.equal(y[~bad], clean[~bad])


RANGE = [(12, 512, 64), (200, 2048, 300), (300, 256, 2048), (64, 4096, 11008), (600, 512, 4400), (4400, 512, 4400),
         (20000, 512, 96), (3, 1000, 50)]
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


@pytest.mark.parametrize("n,cols,units", RANGE)
def test_products_over_the_range_of_scales(n, cols, units):
    """Scale codes from 0 to 252, every pair of them in one product. A row of x holds one value, so that a result is
    one product of two codes and two scales: exact where fp32 holds it, to within its smallest step below the normal
    numbers, infinity above the largest. x from fp32 and bf16 rows as well, whose values are codes as they stand."""
    require_gpu()
    cx = torch.tensor([127, 0, 252, 1, 250, 64, 100, 190, 2, 125, 30, 240])[torch.arange(n) % 12]
    cw = torch.tensor([127, 0, 252, 105, 1, 22, 131, 200, 251, 3, 64, 110, 90])[torch.arange(units) % 13]
    kx, kw = 1 + torch.arange(n) % 7 + 8 * (torch.arange(n) % 5 == 3), 1 + (torch.arange(units) // 13) % 7
    at = (37 * torch.arange(n)) % cols
    (xs, ss), (ws, sw) = tw.mx4_shapes(n, cols), tw.mx4_shapes(units, cols)
    blocks = -(-cols // 32)
    xq, xsc, wsc = torch.zeros(xs, dtype=torch.uint8), torch.zeros(ss, dtype=torch.uint8), torch.zeros(sw, dtype=torch.uint8)
    xq[torch.arange(n), at // 2] = (kx << 4 * (at % 2)).to(torch.uint8)
    xsc[:, :blocks] = cx.to(torch.uint8)[:, None]
    wq = torch.zeros(ws, dtype=torch.uint8)
    wq[:, :cols // 2] = (17 * kw).to(torch.uint8)[:, None]
    wsc[:, :blocks] = cw.to(torch.uint8)[:, None]
    level = torch.tensor(LEVELS, dtype=torch.float64)
    power = lambda c: torch.ldexp(torch.ones(len(c), dtype=torch.float64), c - 127)  # noqa: E731
    xv, wv = level[kx] * power(cx), level[kw] * power(cw)
    want = (xv[:, None] * wv).cuda()
    ops = [v.cuda() for v in (xq, xsc, wq, wsc)]
    x = torch.zeros(n, cols, dtype=torch.float64)
    x[torch.arange(n), at] = xv
    assert torch.equal(x.float().double(), x) and torch.equal(x.to(BF).double(), x)
    top = torch.finfo(F32).max
    assert bool((want.abs() > top).any()) and bool((want.abs() < 2.0 ** -126).any())
    for name, y in (("matmul", tw.matmul_mx4(*ops, cols, dtype=F32)),
                    ("fp32", tw.linear_mx4(x.float().cuda(), *ops[2:], dtype=F32)),
                    ("bf16", tw.linear_mx4(x.to(BF).cuda(), *ops[2:], dtype=F32))):
        print(f"[range] {n}x{cols}x{units} {name}", flush=True)
        y = y.double()
        over, normal = want.abs() > top, want.abs() >= 2.0 ** -126
        assert torch.equal(y[over], torch.copysign(torch.full_like(want[over], float("inf")), want[over]))
        exact = normal & ~over
        assert torch.equal(y[exact], want[exact])
        assert bool(((y - want).abs()[~normal] <= 2.0 ** -149).all())
    # rounded to bf16: the values have four significant bits, so only what fp32 rounds differs
    assert torch.equal(tw.matmul_mx4(*ops, cols), tw.matmul_mx4(*ops, cols, dtype=F32).to(BF))


NORM_WIDTHS = [95, 127, 128, 129, 130, 136, 200, 255, 256, 257, 5003, 8190]


@pytest.mark.parametrize("cols", NORM_WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 21])
def test_norm_widths(rows, cols):
    """Rows of one lane group among several of a wave, with every type; 21 rows leave the last workgroup unfilled."""
    norm.test_forward_widths(rows, cols)


@pytest.mark.parametrize("rows,cols", [(1031, 130), (1027, 200), (2051, 95), (1029, 256), (515, 8190)])
def test_norm_many_rows(rows, cols):
    """The last workgroup of narrow rows is not full."""
    require_gpu()
    for k, (res, delta, out) in enumerate([(BF, F32, BF), (F32, None, F32), (F32, BF, BF), (BF, BF, F32)]):
        norm._forward_case(rows, cols, res, delta, out, BF, seed=3 + k)


BACKWARD = [(37, 95), (5, 127), (1029, 130), (600, 200), (515, 255), (700, 256), (33, 257), (9, 8190), (300, 5003), (517, 999),
            (77, 3001)]


@pytest.mark.parametrize("rows,cols", BACKWARD)
def test_norm_backward(rows, cols):
    norm.test_backward(rows, cols)
