"""The linear layer's products in every tile, split, layout and kind of lines that a call can reach (test_sublayer_cpu.py asks
the library's plans that these sizes do), and every activation and residual in every tile."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw

import linear_reference as lr
from gpu_util import require_gpu
from test_gpu_linear import _gen, _randn, _whole, _ws
from test_gpu_norm import _check_guards, _guarded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# straight from memory: 8, 16, 24 and 32 rows a workgroup, one and several of them, lines of every kind
DIRECT = [(9, 64, 40), (17, 1000, 2049), (30, 520, 1500), (39, 1001, 2100), (50, 999, 2048), (50, 1000, 2048), (70, 2047, 1999),
          (96, 2048, 1000), (90, 5, 1000), (100, 7, 4000), (250, 72, 1100), (24, 5632, 2048), (40, 2048, 4096)]
# rows, k, units of the product
ROWS = DIRECT + [(600, 7, 64), (600, 8, 64), (600, 73, 64), (600, 1000, 64), (600, 1001, 64),
        (33, 7, 64), (33, 8, 64), (33, 73, 64), (33, 1000, 64), (33, 1001, 64), (4100, 8, 500), (1000, 73, 2056), (3000, 2000, 129),
        (2100, 4001, 129), (1500, 200, 4104), (1500, 129, 4104), (300, 8192, 4000), (2000, 131073, 129), (4100, 200, 3000),
        (4353, 1000, 4097), (1500, 8192, 3000), (3000, 2001, 4105), (8000, 513, 8000)]
OTHERS = [(33, 8, 64), (33, 8, 7), (33, 8, 100), (33, 1000, 64), (33, 1000, 100), (1000, 8, 2056), (4100, 8, 500), (4100, 4001, 64),
          (3000, 2000, 129), (1500, 129, 4104), (1500, 129, 4105), (4100, 129, 3000), (3000, 520, 4105), (8000, 8, 4105),
          (300, 8192, 4000), (3000, 32768, 129), (1500, 8192, 3000)]
COLS = OTHERS + [(5632, 512, 2048), (5600, 513, 2056), (5000, 200, 2048), (1000, 32768, 3704)]


@pytest.mark.parametrize("rows,k,units", ROWS)
def test_forward_products(rows, k, units):
    require_gpu()
    gen = _gen(rows + k)
    x, w = _whole(gen, rows, k), _whole(gen, units, k)
    want = x.double() @ w.double().t()
    for y in (F32, BF):
        out, guard = _guarded((rows, units), y)
        ws, wguard = _ws(tw.linear_ws(rows, k, units))
        print(f"[linear] {rows}x{k}x{units} {y}", flush=True)
        tw.linear(x, w, out=out, ws=ws)
        torch.cuda.synchronize()
        _check_guards(guard, wguard)
        assert torch.equal(out, want.to(y))


@pytest.mark.parametrize("rows,k,units", OTHERS)
def test_input_gradient_products(rows, k, units):
    """dx of `rows` tokens, `units` columns and k units."""
    require_gpu()
    gen = _gen(rows + k)
    g, w, x = _whole(gen, rows, k), _whole(gen, k, units), torch.empty(rows, units, dtype=BF, device="cuda")
    want = g.double() @ w.double()
    for t in (F32, BF):
        out, guard = _guarded((rows, units), t)
        ws, wguard = _ws(tw.linear_bwd_ws(rows, units, k, BF, "none", tw.LINEAR_DX))
        print(f"[linear dx] {rows}x{k}x{units} {t}", flush=True)
        tw.linear_bwd(g, x, w, out=(out, None, None), ws=ws)
        torch.cuda.synchronize()
        _check_guards(guard, wguard)
        assert torch.equal(out, want.to(t))


@pytest.mark.parametrize("rows,k,units", COLS)
def test_weight_gradient_products(rows, k, units):
    """dw of `rows` units, `units` columns and k tokens."""
    require_gpu()
    gen = _gen(rows + k)
    g, x, w = _whole(gen, k, rows), _whole(gen, k, units), torch.empty(rows, units, dtype=BF, device="cuda")
    want = g.double().t() @ x.double()
    for t in (F32, BF):
        out, guard = _guarded((rows, units), t)
        ws, wguard = _ws(tw.linear_bwd_ws(k, units, rows, BF, "none", tw.LINEAR_DW))
        print(f"[linear dw] {rows}x{k}x{units} {t}", flush=True)
        tw.linear_bwd(g, x, w, out=(None, out, None), ws=ws)
        torch.cuda.synchronize()
        _check_guards(guard, wguard)
        assert torch.equal(out, want.to(t))


# tokens, columns, units whose two products run in one launch (host_check_sublayer.cpp asks that they do), the last ones
# nearly as many tiles as run at a time
PAIRS = [(1, 8, 1), (33, 100, 100), (64, 128, 64), (65, 129, 63), (1, 4096, 500), (500, 1000, 9), (509, 1000, 1021), (509, 1021, 1000),
         (2049, 264, 500), (2000, 1001, 2000), (2048, 1024, 2048)]


@pytest.mark.parametrize("n,cols,units", PAIRS)
@pytest.mark.parametrize("dx_type,dw_type", [(BF, F32), (F32, BF)])
def test_both_gradient_products_at_a_time(n, cols, units, dx_type, dw_type):
    require_gpu()
    gen = _gen(n + cols)
    g, x, w = _whole(gen, n, units), _whole(gen, n, cols), _whole(gen, units, cols)
    (dx, a), (dw, b), (db, c) = _guarded((n, cols), dx_type), _guarded((units, cols), dw_type), _guarded((units,), F32)
    ws, d = _ws(tw.linear_bwd_ws(n, cols, units, BF, "none"))
    print(f"[linear bwd] {n}x{cols}x{units} {dx_type} {dw_type}", flush=True)
    tw.linear_bwd(g, x, w, out=(dx, dw, db), ws=ws)
    torch.cuda.synchronize()
    _check_guards(a, b, c, d)
    assert torch.equal(dx, (g.double() @ w.double()).to(dx_type))
    assert torch.equal(dw, (g.double().t() @ x.double()).to(dw_type))
    assert torch.equal(db, g.double().sum(0).float())


# one size for each tile, of aligned lines and of lines at any element
EPILOGUES = [(50, 72, 2056), (70, 73, 2001), (600, 72, 200), (600, 73, 203), (33, 72, 200), (100, 73, 203), (1000, 72, 2056), (1000, 73, 2059), (1500, 200, 4104), (1500, 129, 4103), (4100, 200, 3000)]


@pytest.mark.parametrize("rows,cols,units", EPILOGUES)
@pytest.mark.parametrize("act", list(tw.ACTS))
def test_epilogues(rows, cols, units, act):
    require_gpu()
    for k, (bias, res, y) in enumerate(((None, None, BF), (F32, F32, BF), (BF, BF, F32), (BF, None, F32), (None, BF, BF))):
        gen = _gen(k)
        x, w = _randn(gen, rows, cols, dtype=BF), _randn(gen, units, cols, scale=2 / cols ** 0.5, dtype=BF)
        b = None if bias is None else _randn(gen, units, scale=2, dtype=bias)
        r = None if res is None else _randn(gen, rows, units, dtype=res)
        (z, tz), (want, tol) = lr.forward(x, w, b, act, r, y)
        pre, pguard = _guarded((rows, units), BF)
        out, guard = _guarded((rows, units), y)
        print(f"[linear] {rows}x{cols}x{units} {act} {bias} {res} {y}", flush=True)
        tw.linear(x, w, bias=b, act=act, residual=r, out=out, pre=pre)
        torch.cuda.synchronize()
        _check_guards(guard, pguard)
        assert bool(((out.double() - want).abs() <= tol).all())
        assert bool(((pre.double() - z).abs() <= lr.rounded(tz, z, BF)).all())
        if res == y:
            tw.linear(x, w, bias=b, act=act, residual=r, out=r)
            assert torch.equal(r, out)


def test_results_beyond_32_bits_of_elements():
    """More than 2^31 results and operands' elements; rows, columns and corners against float64."""
    require_gpu()
    rows, cols, units = (1 << 20) + 200, 72, 2304
    gen = _gen(1)
    x, w = _whole(gen, rows, cols), _whole(gen, units, cols)
    y = tw.linear(x, w)
    assert y.numel() > 1 << 31
    for part in (slice(0, 300), slice((1 << 31) // units - 200, (1 << 31) // units + 200), slice(rows - 300, rows)):
        assert torch.equal(y[part], (x[part].double() @ w.double().t()).to(BF))
    dx = tw.linear_bwd(y, x, w, out=(torch.empty_like(x), None, None)).dx
    for part in (slice(0, 300), slice((1 << 31) // units - 200, (1 << 31) // units + 200), slice(rows - 300, rows)):
        got, want = dx[part].double(), y[part].double() @ w.double()
        tol = (y[part].double().abs() @ w.double().abs()) * units * lr.U
        assert bool(((got - want).abs() <= lr.rounded(tol, want, BF)).all())


def test_weights_of_more_elements_than_a_launch_writes():
    """A weight's gradient of no rows, of more than 2^32 pieces of 8: zeros in its first and last rows and around the border
    of two launches."""
    require_gpu()
    units, cols = (1 << 18) + 3, (1 << 17) + 4
    pieces = (cols + 7) // 8
    assert units * pieces > 1 << 32
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of free device memory")
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    x, w, dw = e(0, cols), e(units, cols), e(units, cols).fill_(3)
    tw.linear_bwd(e(0, units), x, w, out=(None, dw, None))
    border = ((1 << 32) - 256) // pieces
    for part in (slice(0, 9), slice(border - 9, border + 9), slice(units - 9, units)):
        assert not dw[part].any()
    del w, dw
    torch.cuda.empty_cache()
