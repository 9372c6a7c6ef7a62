"""Refusals of the operators around the block: the C ABI before it touches a device, and the Python binding before it
hands an address over. Needs no GPU; the addresses are never read."""
import ctypes

import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)
EPS = ctypes.c_float(1e-6)


def _norm(rows=4, cols=64, rt=0, r=FAKE, dt=0, d=None, wt=0, w=FAKE, eps=EPS, ro=FAKE, ot=0, o=FAKE, q=None, qs=None,
          rstd=None):
    return tw.lib().twell_add_rms_norm(rows, cols, rt, r, dt, d, wt, w, eps, ro, ot, o, q, qs, rstd, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), 1, b"rows"), (dict(cols=0), 1, b"cols"), (dict(cols=16385), 2, b"16384"),
    (dict(rows=1 << 31), 2, b"rows"), (dict(rt=2), 1, b"dtypes"), (dict(wt=-1), 1, b"dtypes"), (dict(ot=5), 1, b"dtypes"),
    (dict(d=FAKE, dt=9), 1, b"dtypes"), (dict(eps=ctypes.c_float(0)), 1, b"eps"),
    (dict(eps=ctypes.c_float(-1e-6)), 1, b"eps"), (dict(eps=ctypes.c_float(float("nan"))), 1, b"eps"),
    (dict(eps=ctypes.c_float(float("inf"))), 1, b"eps"), (dict(r=None), 1, b"residual"), (dict(r=ODD), 1, b"residual"),
    (dict(w=None), 1, b"weight"), (dict(d=ODD), 1, b"delta"), (dict(ro=ODD), 1, b"residual_out"), (dict(o=ODD), 1, b"out"),
    (dict(q=FAKE), 1, b"q_scale"), (dict(q=ODD, qs=FAKE), 1, b"q"), (dict(rstd=ODD), 1, b"rstd"),
    (dict(ro=None, o=None), 1, b"no output"),
])
def test_norm_refusals(kw, code, word):
    assert _norm(**kw) == code
    assert word in tw.lib().twell_last_error()


def test_norm_of_no_rows_needs_no_device():
    assert _norm(rows=0, r=None, ro=None, o=None) == 0
    assert tw.lib().twell_last_error() == b""


def _bwd(rows=600, cols=64, gt=0, g=FAKE, rt=0, ds=None, r=FAKE, rstd=FAKE, wt=0, w=FAKE, dr=FAKE, dw=FAKE, ws=FAKE,
         n=1 << 20):
    return tw.lib().twell_add_rms_norm_bwd(rows, cols, gt, g, rt, ds, r, rstd, wt, w, dr, dw, ws, n, None)


def test_norm_backward_workspace():
    assert tw.add_rms_norm_bwd_ws(4, 64) == 0          # one workgroup writes dw itself
    assert tw.add_rms_norm_bwd_ws(600, 64) == 38 * 64 * 4
    assert tw.add_rms_norm_bwd_ws(600, 4096) == 256 * 4096 * 4
    with pytest.raises(tw.TwellError):
        tw.add_rms_norm_bwd_ws(4, 20000)
    assert tw.lib().twell_add_rms_norm_bwd_ws(4, 64, None) == 1


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), 1, b"rows"), (dict(cols=16385), 2, b"16384"), (dict(gt=3), 1, b"dtypes"), (dict(g=None), 1, b"d_out"),
    (dict(ds=ODD), 1, b"d_residual"), (dict(r=None), 1, b"residual"), (dict(rstd=None), 1, b"rstd"),
    (dict(w=None), 1, b"weight"), (dict(dr=None), 1, b"dr"), (dict(dw=ODD), 1, b"dw"),
    (dict(n=38 * 64 * 4 - 1), 3, b"workspace"), (dict(ws=None), 3, b"workspace"), (dict(ws=ODD), 3, b"workspace"),
])
def test_norm_backward_refusals(kw, code, word):
    assert _bwd(**kw) == code
    assert word in tw.lib().twell_last_error()


def test_binding_refuses_what_does_not_fit():
    r, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        tw.add_rms_norm(r, w)
    with pytest.raises(ValueError, match="rows, cols"):
        tw.add_rms_norm(r[0], w)
    with pytest.raises(TypeError, match="residual"):
        tw.add_rms_norm(r.half(), w)
    with pytest.raises(ValueError, match="codes and scale"):
        tw.add_rms_norm(r, w, out=(None, r, torch.zeros(4, 64, dtype=torch.uint8), None, None))
    with pytest.raises(ValueError, match="rows, cols"):
        tw.add_rms_norm_bwd(r, r[0], r[0], w)
    with pytest.raises(ValueError, match="GPU"):
        tw.add_rms_norm_bwd(r, r, r[:, 0].contiguous(), w)
    f = tw._addr
    with pytest.raises(ValueError, match="shape"):
        f(r, "x", (4, 63))
    with pytest.raises(TypeError, match="uint8"):
        f(r, "x", (4, 64), torch.uint8)
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(64, 4).t(), "x", (4, 64))
    assert f(None, "x", (4, 64)) is None


# ---------------------------------------------------------------- MX4

def _sizes(rows, cols):
    q, s = ctypes.c_size_t(), ctypes.c_size_t()
    st = tw.lib().twell_mx4_sizes(rows, cols, ctypes.byref(q), ctypes.byref(s))
    return st, q.value, s.value


def test_mx4_sizes_and_shapes():
    for rows, cols in ((1, 1), (3, 128), (3, 129), (7, 512), (7, 513), (11008, 4096), (0, 64)):
        st, q, s = _sizes(rows, cols)
        (r0, c0), (r1, c1) = tw.mx4_shapes(rows, cols)
        assert st == 0 and (q, s) == (r0 * c0, r1 * c1)
        assert 2 * c0 >= cols and 32 * c1 >= cols and c0 % 64 == 0 and c1 % 16 == 0
    assert _sizes(-1, 64)[0] == 1 and _sizes(1, 0)[0] == 1 and _sizes(1, (1 << 20) + 1)[0] == 2
    assert _sizes(1 << 31, 64)[0] == 2 and _sizes((1 << 31) - 1, 1 << 20)[0] == 2
    assert tw.lib().twell_mx4_sizes(1, 64, None, None) == 1


def test_mx4_product_workspaces():
    """Nothing for few tokens, x's MX4 rows for some more, and for tiles both operands' scales by 256 columns (8 bytes
    a row, 128 rows at least) in place of x's scale rows."""
    assert tw.linear_mx4_ws(1, 4096, 11008) == 0 and tw.linear_mx4_ws(0, 4096, 11008) == 0
    assert tw.linear_mx4_ws(24, 2048, 5632) == 0 and tw.linear_mx4_ws(200, 512, 1024) == 0
    assert tw.linear_mx4_ws(30, 1990, 8100) == 30 * (1024 + 64) and tw.matmul_mx4_ws(30, 1990, 8100) == 0
    assert tw.linear_mx4_ws(1000, 1990, 100) == 1000 * (1024 + 64)  # fewer units than a tile
    assert tw.linear_mx4_ws(100, 200, 30000) == 100 * (128 + 16)    # fewer tokens than a tile, and one stage of columns
    assert tw.linear_mx4_ws(1000, 200, 8100) == 1000 * 128 + 8 * (8100 + 1000)
    arranged = 8 * 8 * (8100 + 1000)
    assert tw.linear_mx4_ws(1000, 1990, 8100) == 1000 * 1024 + arranged and tw.matmul_mx4_ws(1000, 1990, 8100) == arranged
    # fewer tokens than a tile: x's scales are given a tile's rows
    assert tw.matmul_mx4_ws(100, 4096, 11008) == 16 * 8 * (11008 + 128)
    assert tw.matmul_mx4_ws(100, 1000, 1000) == 0  # too little work for tiles
    for f in (tw.lib().twell_linear_mx4_ws, tw.lib().twell_matmul_mx4_ws):
        assert f(1, 64, 8, None) == 1
        n = ctypes.c_size_t()
        assert f(1, 64, 0, ctypes.byref(n)) == 1 and f(-1, 64, 8, ctypes.byref(n)) == 1 and f(1, 1 << 21, 8, ctypes.byref(n)) == 2


def test_mx4_refusals():
    L = tw.lib()
    q = lambda rows=4, cols=64, dt=0, a=FAKE, c=FAKE, s=FAKE: L.twell_quantize_mx4(rows, cols, dt, a, c, s, None)  # noqa: E731
    assert q(rows=-1) == 1 and q(cols=0) == 1 and q(cols=1 << 21) == 2 and q(dt=4) == 1
    assert q(a=None) == 1 and q(c=ODD) == 1 and q(s=None) == 1 and b"scale" in L.twell_last_error()
    d = lambda rows=4, cols=64, c=FAKE, s=FAKE, dt=0, o=FAKE: L.twell_dequantize_mx4(rows, cols, c, s, dt, o, None)  # noqa: E731
    assert d(rows=-1) == 1 and d(c=None) == 1 and d(s=ODD) == 1 and d(dt=2) == 1 and d(o=None) == 1
    m = lambda n=4, k=64, u=8, a=FAKE, b=FAKE, c=FAKE, e=FAKE, dt=0, y=FAKE, ws=None, b2=0: L.twell_matmul_mx4(  # noqa: E731
        n, k, u, a, b, c, e, dt, y, ws, b2, None)
    for kw in (dict(n=-1), dict(k=0), dict(u=0), dict(a=None), dict(b=ODD), dict(c=None), dict(e=None), dict(dt=3), dict(y=None)):
        assert m(**kw) == 1, kw
    assert m(u=(1 << 24) + 1) == 2 and m(n=(1 << 31) - 1, u=1 << 20) == 2
    need = 16 * 8 * (11008 + 128)
    tiles = dict(n=100, k=4096, u=11008)
    assert m(**tiles) == 3 and m(**tiles, ws=FAKE, b2=need - 1) == 3
    assert m(**tiles, ws=ODD, b2=need) == 3 and b"workspace" in L.twell_last_error()
    f = lambda n=64, k=4096, u=8, xd=0, x=FAKE, c=FAKE, e=FAKE, dt=0, y=FAKE, ws=FAKE, b=64 * 2176: L.twell_linear_mx4(  # noqa: E731
        n, k, u, xd, x, c, e, dt, y, ws, b, None)
    for kw in (dict(xd=9), dict(x=None), dict(x=ODD), dict(c=None), dict(y=ODD)):
        assert f(**kw) == 1, kw
    assert tw.linear_mx4_ws(64, 4096, 8) == 64 * 2176
    assert f(b=64 * 2176 - 1) == 3 and f(ws=None) == 3 and f(ws=ODD) == 3


def test_mx4_of_no_rows_needs_no_device():
    L = tw.lib()
    assert L.twell_quantize_mx4(0, 64, 0, None, None, None, None) == 0
    assert L.twell_dequantize_mx4(0, 64, None, None, 0, None, None) == 0
    assert L.twell_matmul_mx4(0, 64, 8, None, None, FAKE, FAKE, 0, None, None, 0, None) == 0
    assert L.twell_linear_mx4(0, 64, 8, 0, None, FAKE, FAKE, 0, None, None, 0, None) == 0


def test_mx4_binding_refuses_what_does_not_fit():
    x = torch.zeros(4, 64)
    w = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 16, dtype=torch.uint8)
    for call in (lambda: tw.quantize_mx4(x), lambda: tw.linear_mx4(x, *w), lambda: tw.dequantize_mx4(*w, 64),
                 lambda: tw.matmul_mx4(*w, *w, 64)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="rows, cols"):
        tw.quantize_mx4(x[0])
    with pytest.raises(TypeError, match="bfloat16"):
        tw.quantize_mx4(x.half())
    with pytest.raises(ValueError, match="rows, cols"):
        tw.linear_mx4(x[0], *w)
    with pytest.raises(ValueError, match="shape"):
        tw.dequantize_mx4(*w, 200)


def test_serve_refuses_settings():
    dims = tw.make_dims(1, 64, 128, 64, 64)
    with pytest.raises(ValueError, match="gate"):
        tw.TwellServe(dims, "int4", device="cpu")
    with pytest.raises(ValueError, match="stream"):
        tw.TwellServe(dims, "mx4", stream_dtype=torch.float16, device="cpu")
    s = tw.TwellServe(tw.make_dims(128, 4096, 256, 64, 8, 0, 16), "mx4", device="cpu")
    assert not s.capture_supported()  # as the bf16 gate at this size
    with pytest.raises(tw.TwellError, match="capture"):
        s.capture(None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        s.forward(torch.zeros(128, 4096, dtype=torch.bfloat16), None, None, None,
                  *[torch.zeros(256, 4096, dtype=torch.bfloat16)] * 2, torch.zeros(128))
