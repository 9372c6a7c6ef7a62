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
    assert tw.add_rms_norm_bwd_ws(600, 64) == 150 * 64 * 4
    assert tw.add_rms_norm_bwd_ws(600, 4096) == 512 * 4096 * 4
    with pytest.raises(tw.TwellError):
        tw.add_rms_norm_bwd_ws(4, 20000)
    assert tw.lib().twell_add_rms_norm_bwd_ws(4, 64, None) == 1


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), 1, b"rows"), (dict(cols=16385), 2, b"16384"), (dict(gt=3), 1, b"dtypes"), (dict(g=None), 1, b"d_out"),
    (dict(ds=ODD), 1, b"d_residual"), (dict(r=None), 1, b"residual"), (dict(rstd=None), 1, b"rstd"),
    (dict(w=None), 1, b"weight"), (dict(dr=None), 1, b"dr"), (dict(dw=ODD), 1, b"dw"),
    (dict(n=150 * 64 * 4 - 1), 3, b"workspace"), (dict(ws=None), 3, b"workspace"), (dict(ws=ODD), 3, b"workspace"),
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
