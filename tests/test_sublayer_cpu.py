"""What holds for the linear layer, the join and dropout without a GPU: the generator against published vectors, the oracles'
gradients against differences, refusals of the C ABI and of the binding, devices and streams, the kernels that the GPU tests'
sizes reach, waits in front of loads into LDS."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import join_reference as jr
import linear_reference as lr
import test_gpu_linear_variants as variants
from activation_sparse_ffn_03_amd import build as b
from activation_sparse_ffn_03_amd import twell as tw
from test_host_sanitize import CSRC, ROOT, _rocm
from test_lds_load_wait_cpu import _listing, hazards
from test_ops_binding_cpu import _OnGpu, _Stream, library  # noqa: F401

CSRC_OPS = os.path.join(ROOT, "activation_sparse_ffn_03_amd", "csrc_ops")
BF, F32, U8, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64
FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)


# ---------------------------------------------------------------- generator and oracles

@pytest.mark.parametrize("counter,key,block", [
    ((0,) * 4, (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((jr.M32,) * 4, (jr.M32,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_vectors(counter, key, block):
    """The vectors that Philox4x32-10 was published with."""
    assert tuple(int(v) for v in jr.philox(counter, key)) == block


def test_mask_of_a_part_is_the_part_of_the_mask():
    whole = jr.kept(40, 77, 0.3, 12345, 6, 7)
    assert torch.equal(jr.kept(10, 77, 0.3, 12345, 6, 7, 20), whole[20:30])
    assert torch.equal(jr.kept(40, 16, 0.3, 12345, 6, 7), whole[:, :16])
    assert jr.threshold(0.0) == 0 and jr.threshold(1.0) == 65536 and jr.factor(1.0) == 0 and jr.factor(0.5) == 2


def _differences(f, tensors, grads, step=1e-6):
    """Every gradient entry (a few of each) against a central difference of f in float64."""
    for t, g in zip(tensors, grads):
        if t is None:
            continue
        flat = t.reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
            old = float(flat[i])
            flat[i] = old + step
            up = f()
            flat[i] = old - step
            dn = f()
            flat[i] = old
            d = (up - dn) / (2 * step)
            # the third derivative's step^2 and cancellation's 1e-15 / step of sums below 100
            assert abs(d - float(g.reshape(-1)[i])) <= 1e-6 * (1 + abs(d))


@pytest.mark.parametrize("post,gates,p", [(True, 3, 0.3), (True, 0, 0.0), (False, 6, 0.2), (False, 1, 0.0)])
def test_join_oracle_gradient(post, gates, p):
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    rows, cols, eps, alpha = 6, 20, 1e-6, 0.75
    r, y, w, pw = rnd(rows, cols), rnd(rows, cols), 1 + 0.3 * rnd(cols), 1 + 0.3 * rnd(cols)
    gate = rnd(gates, cols) if gates else None
    d_out, d_res = rnd(rows, cols), rnd(rows, cols)
    keep = jr.kept(rows, cols, p, 5, 6, 7) if p else None
    pw = pw if post else None

    def forward():
        st, ry = jr.stream64(r, y, pw, gate, alpha, eps, keep, p)
        rho = 1 / torch.sqrt((st * st).mean(1, keepdim=True) + eps)
        return st, rho, ry

    def loss():
        st, rho, _ = forward()
        return float((st * rho * w * d_out).sum() + (st * d_res).sum())

    st, rho, ry = forward()
    grads = jr.backward64(d_out, d_res, st, rho, y, ry, w, pw, gate, alpha, keep, p)
    _differences(loss, [r, y, w, pw, gate], grads)


@pytest.mark.parametrize("act", list(tw.ACTS))
def test_linear_oracle_gradient(act):
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, bias, g = rnd(5, 7), rnd(6, 7), rnd(6), rnd(5, 6)
    f = lambda: float((lr.act64(x @ w.t() + bias, act) * g).sum())  # noqa: E731
    grads = [v for v, _ in lr.backward(g, x, w, act, x @ w.t() + bias, F32, F32)]
    _differences(f, [x, w, bias], grads)


# ---------------------------------------------------------------- refusals of the C ABI

def _dropout(rows=4, cols=64, t=0, x=FAKE, p=0.5, rng=FAKE, site=0, out=FAKE):
    return tw.lib().twell_dropout(rows, cols, t, x, p, rng, site, out, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), 1, b"rows"), (dict(cols=0), 1, b"cols"), (dict(rows=1 << 31), 2, b"rows"), (dict(cols=(1 << 30) + 1), 2, b"cols"),
    (dict(t=2), 1, b"dtypes"), (dict(p=-0.1), 1, b"p must"), (dict(p=1.1), 1, b"p must"), (dict(p=float("nan")), 1, b"p must"),
    (dict(x=None), 1, b"x"), (dict(out=ODD), 1, b"out"), (dict(rng=None), 1, b"rng"), (dict(rng=ODD), 1, b"rng"),
    (dict(rng=None, p=0.0), 1, b"rng"), (dict(rng=ODD, p=0.0), 1, b"rng")])
def test_dropout_refusals(kw, code, word):
    assert _dropout(**kw) == code
    assert word in tw.lib().twell_last_error()


def _options(**kw):
    d = dict(post_weight=FAKE, gate=FAKE, rng=FAKE, gate_rows=2, alpha=1.0, p=0.25, site=0, post_weight_dtype=0, gate_dtype=0)
    d.update(kw)
    return tw.Join(**{k: (v.value if isinstance(v, ctypes.c_void_p) else v) for k, v in d.items()})


def _join(rows=4, cols=64, rt=0, r=FAKE, yt=0, y=FAKE, wt=0, w=FAKE, eps=1e-6, ro=FAKE, ot=0, o=FAKE, q=None, qs=None, rstd=None,
          prstd=None, j=None, **opt):
    return tw.lib().twell_join_rms_norm(rows, cols, rt, r, yt, y, wt, w, _options(**opt) if j is None else j, eps, ro, ot, o, q, qs,
                                        rstd, prstd, None)


BAD_OPTIONS = [
    (dict(gate_rows=0), 1, b"gate_rows"), (dict(gate_rows=3), 1, b"gate_rows"), (dict(gate_rows=-1), 1, b"gate_rows"),
    (dict(gate_rows=8), 1, b"gate_rows"), (dict(gate=ODD), 1, b"gate"), (dict(gate_dtype=4), 1, b"dtypes"),
    (dict(post_weight=ODD), 1, b"post_weight"), (dict(post_weight_dtype=-1), 1, b"dtypes"), (dict(alpha=float("inf")), 1, b"alpha"),
    (dict(alpha=float("nan")), 1, b"alpha"), (dict(p=-1e-3), 1, b"p must"), (dict(p=1.5), 1, b"p must"), (dict(rng=None), 1, b"rng"),
    (dict(rng=ODD), 1, b"rng"), (dict(rows=-1), 1, b"rows"), (dict(cols=0), 1, b"cols"), (dict(cols=16385), 2, b"16384"),
    (dict(rows=1 << 31), 2, b"rows"), (dict(rt=2), 1, b"dtypes"), (dict(yt=3), 1, b"dtypes"), (dict(wt=-1), 1, b"dtypes"),
    (dict(r=None), 1, b"residual"), (dict(y=ODD), 1, b"y"), (dict(w=None), 1, b"weight")]


@pytest.mark.parametrize("kw,code,word", BAD_OPTIONS + [
    (dict(ot=5), 1, b"dtypes"), (dict(eps=0.0), 1, b"eps"), (dict(eps=float("nan")), 1, b"eps"), (dict(ro=ODD), 1, b"residual_out"),
    (dict(o=ODD), 1, b"out"), (dict(q=FAKE), 1, b"q_scale"), (dict(rstd=ODD), 1, b"rstd"), (dict(prstd=ODD), 1, b"post_rstd"),
    (dict(prstd=FAKE, post_weight=None), 1, b"post_rstd"), (dict(ro=None, o=None), 1, b"no output")])
def test_join_refusals(kw, code, word):
    assert _join(**kw) == code
    assert word in tw.lib().twell_last_error()


def test_join_without_its_options_is_refused():
    assert tw.lib().twell_join_rms_norm(4, 64, 0, FAKE, 0, FAKE, 0, FAKE, None, 1e-6, FAKE, 0, FAKE, None, None, None, None, None) == 1
    assert b"join" in tw.lib().twell_last_error()


def _join_bwd(rows=600, cols=64, gt=0, g=FAKE, rt=0, ds=None, r=FAKE, rstd=FAKE, yt=0, y=FAKE, prstd=FAKE, wt=0, w=FAKE, dr=FAKE,
              dy=FAKE, dw=FAKE, dp=FAKE, dg=FAKE, ws=FAKE, n=1 << 30, **opt):
    return tw.lib().twell_join_rms_norm_bwd(rows, cols, gt, g, rt, ds, r, rstd, yt, y, prstd, wt, w, _options(**opt), dr, dy, dw, dp, dg,
                                            ws, n, None)


@pytest.mark.parametrize("kw,code,word", [(k, c, w) for k, c, w in BAD_OPTIONS if k not in (dict(gate_rows=3), dict(gate_rows=8))] + [
    (dict(gate_rows=7), 1, b"gate_rows"), (dict(gt=2), 1, b"dtypes"), (dict(g=None), 1, b"d_out"), (dict(ds=ODD), 1, b"d_residual"),
    (dict(rstd=None), 1, b"rstd"), (dict(prstd=None), 1, b"post_rstd"), (dict(dr=None), 1, b"dr"), (dict(dy=ODD), 1, b"dy"),
    (dict(dw=None), 1, b"dw"), (dict(dp=None), 1, b"dpost"), (dict(dg=None), 1, b"dgate"), (dict(n=8), 3, b"workspace"),
    (dict(ws=None), 3, b"workspace"), (dict(ws=ODD), 3, b"workspace")])
def test_join_backward_refusals(kw, code, word):
    assert _join_bwd(**kw) == code
    assert word in tw.lib().twell_last_error()


def test_join_backward_workspace():
    assert tw.join_rms_norm_bwd_ws(2, 64, True, 0) == 0                       # one workgroup writes the sums itself
    assert tw.join_rms_norm_bwd_ws(0, 64, True, 5) == 0
    assert tw.join_rms_norm_bwd_ws(8192, 2048, True, 1) == 3 * 256 * 2048 * 4  # dw, dpost and the gate's partial rows
    assert tw.join_rms_norm_bwd_ws(8192, 2048, False, 0) == 256 * 2048 * 4
    assert tw.join_rms_norm_bwd_ws(8192, 2048, True, 8192) == 2 * 256 * 2048 * 4  # a gate a row: no sums
    for bad in ((4, 20000, True, 0), (4, 64, True, 3), (-1, 64, True, 0), (4, 64, True, -1)):
        with pytest.raises(tw.TwellError):
            tw.join_rms_norm_bwd_ws(*bad)
    assert tw.lib().twell_join_rms_norm_bwd_ws(4, 64, 1, 0, None) == 1


def _linear(n=100, cols=64, units=32, x=FAKE, w=FAKE, bt=0, bias=FAKE, act=0, rt=0, res=FAKE, pre=None, yt=0, y=ctypes.c_void_p(0x200000),
            ws=FAKE, nb=1 << 30):
    return tw.lib().twell_linear(n, cols, units, x, w, bt, bias, act, rt, res, pre, yt, y, ws, nb, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=-1), 1, b"n must"), (dict(cols=0), 1, b"cols"), (dict(units=-3), 1, b"units"), (dict(cols=(1 << 20) + 1), 2, b"2^20"),
    (dict(units=(1 << 20) + 1), 2, b"2^20"), (dict(n=1 << 31), 2, b"pieces"), (dict(n=1 << 30, units=64), 2, b"pieces"),
    (dict(yt=2), 1, b"dtypes"), (dict(bt=2), 1, b"dtypes"), (dict(rt=-1), 1, b"dtypes"), (dict(act=4), 1, b"act"), (dict(act=-1), 1, b"act"),
    (dict(x=None), 1, b"x"), (dict(w=ODD), 1, b"w"), (dict(bias=ODD), 1, b"bias"), (dict(res=ODD), 1, b"residual"), (dict(pre=ODD), 1, b"pre"),
    (dict(y=None), 1, b"y"), (dict(y=FAKE, rt=1), 1, b"one type"), (dict(n=100, cols=1 << 16, nb=0), 3, b"workspace"),
    (dict(n=100, cols=1 << 16, ws=None), 3, b"workspace"), (dict(n=100, cols=1 << 16, ws=ODD), 3, b"workspace")])
def test_linear_refusals(kw, code, word):
    assert _linear(**kw) == code
    assert word in tw.lib().twell_last_error()


def _linear_bwd(n=100, cols=64, units=32, gt=0, g=FAKE, act=1, pre=FAKE, x=FAKE, w=FAKE, xt=0, dx=FAKE, wt=0, dw=FAKE, db=FAKE, ws=FAKE,
                nb=1 << 30):
    return tw.lib().twell_linear_bwd(n, cols, units, gt, g, act, pre, x, w, xt, dx, wt, dw, db, ws, nb, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=-1), 1, b"n must"), (dict(units=0), 1, b"units"), (dict(cols=1 << 21), 2, b"2^20"), (dict(gt=2), 1, b"dtypes"),
    (dict(xt=2), 1, b"dtypes"), (dict(wt=2), 1, b"dtypes"), (dict(act=9), 1, b"act"), (dict(g=None), 1, b"d_out"), (dict(pre=None), 1, b"pre"),
    (dict(pre=ODD), 1, b"pre"), (dict(x=None), 1, b"x"), (dict(w=None), 1, b"w"), (dict(dx=ODD), 1, b"dx"), (dict(dw=ODD), 1, b"dw"),
    (dict(db=ODD), 1, b"db"), (dict(dx=None, dw=None, db=None), 1, b"no output"), (dict(nb=0), 3, b"workspace"), (dict(ws=None), 3, b"workspace"),
    (dict(ws=ODD), 3, b"workspace")])
def test_linear_backward_refusals(kw, code, word):
    assert _linear_bwd(**kw) == code
    assert word in tw.lib().twell_last_error()


def _apart(call, outputs, inputs, may=(), **given):
    """Each output that begins where an input or an output before it does, or 16 bytes behind, is refused; `may` are pairs that
    may be one and the same array."""
    at = {name: 0x1000000 * (i + 1) for i, name in enumerate((*outputs, *inputs))}
    address = lambda **moved: {n: ctypes.c_void_p(moved.get(n, a)) for n, a in at.items()}  # noqa: E731
    for i, out in enumerate(outputs):
        for other in (*inputs, *outputs[:i]):
            for shift in (0, 16):
                if shift == 0 and (out, other) in may:
                    continue
                assert call(**{**given, **address(**{out: at[other] + shift})}) == 1, (out, other, shift)
                assert b"overlap" in tw.lib().twell_last_error(), (out, other, shift)


def test_outputs_that_overlap_are_refused():
    _apart(_dropout, ["out"], ["x"], [("out", "x")])
    assert _dropout(rng=ctypes.c_void_p(0x2000000), out=ctypes.c_void_p(0x2000000)) == 1
    _apart(_join, ["ro", "o", "q", "rstd", "prstd"], ["r", "y", "w", "post_weight", "gate"], [("ro", "r")], rows=64,
           qs=ctypes.c_void_p(0xF0000000))
    _apart(_join_bwd, ["dr", "dy", "dw", "dp", "dg", "ws"], ["g", "ds", "r", "rstd", "y", "prstd", "w", "post_weight", "gate"])
    _apart(_linear, ["y", "pre", "ws"], ["x", "w", "bias", "res"], [("y", "res")], n=600, cols=1 << 10)
    _apart(_linear_bwd, ["dx", "dw", "db", "ws"], ["g", "pre", "x", "w"])


def test_calls_of_no_rows_need_no_device():
    for st in (_dropout(rows=0, x=None, out=None), _join(rows=0, r=None, y=None, ro=None, o=None, gate_rows=5),
               _linear(n=0, x=None, res=None, y=None, ws=None, nb=0), _linear_bwd(n=0, g=None, pre=None, x=None, dx=None, dw=None, db=None)):
        assert st == 0 and tw.lib().twell_last_error() == b""


def test_workspace_queries():
    assert tw.linear_ws(1, 4096, 11008) == 0 and tw.linear_ws(0, 64, 64) == 0  # straight from memory; nothing
    assert tw.linear_ws(16384, 4096, 11008) == 0
    assert tw.linear_ws(300, 8192, 700) > 0  # splits' sums
    assert tw.linear_bwd_ws(1024, 64, 64, BF, "none", tw.LINEAR_DB) == 0
    assert tw.linear_bwd_ws(8192, 64, 64, BF, "relu", tw.LINEAR_DB) == 64 * 64 * 4  # the bias's partial sums
    assert tw.linear_bwd_ws(100, 64, 64, BF, "relu") > tw.linear_bwd_ws(100, 64, 64, BF, "none")  # dz
    far = (1 << 32) + 64
    for call in (lambda: tw.linear_ws(100, far, 64), lambda: tw.linear_ws(100, 64, far), lambda: tw.linear_bwd_ws(100, far, 64),
                 lambda: tw.linear_bwd_ws(100, 64, far), lambda: tw.join_rms_norm_bwd_ws(100, far, True, 0)):
        with pytest.raises(tw.TwellError, match="UNSUPPORTED"):
            call()
    assert tw.lib().twell_linear_ws(4, 64, 64, None) == 1 and tw.lib().twell_linear_bwd_ws(4, 64, 64, 0, 0, 7, None) == 1


# ---------------------------------------------------------------- the binding

def test_binding_refuses_what_does_not_fit():
    r, w, x = torch.zeros(4, 64), torch.ones(64), torch.zeros(4, 64, dtype=BF)
    rng = torch.zeros(2, dtype=I64)
    for call, err, word in (
            (lambda: tw.dropout(r[0], rng, 0.5), ValueError, "rows, cols"), (lambda: tw.dropout(r.half(), rng, 0.5), TypeError, "x must"),
            (lambda: tw.dropout(r, rng, 0.5), ValueError, "GPU"),
            (lambda: tw.join_rms_norm(r[0], r, w), ValueError, "rows, cols"), (lambda: tw.join_rms_norm(r, r, w), ValueError, "GPU"),
            (lambda: tw.join_rms_norm(r, r, w, out=(r, r, r, None, None, None)), ValueError, "codes and scale"),
            (lambda: tw.join_rms_norm_bwd(r, r[0], w, r, w), ValueError, "rows, cols"),
            (lambda: tw.linear(x[0], x), ValueError, "rows, cols"), (lambda: tw.linear(x, x, act="tanh"), ValueError, "act"),
            (lambda: tw.linear(r, x), TypeError, "bfloat16"), (lambda: tw.linear(x, x), ValueError, "GPU"),
            (lambda: tw.linear_bwd(x, x, x, act="relu"), ValueError, "pre"), (lambda: tw.linear_bwd(x, x[0], x), ValueError, "rows, cols")):
        with pytest.raises(err, match=word):
            call()
    for site in (-1, 1 << 32):
        with pytest.raises(ValueError, match="site"):
            tw._site(site)


def _calls():
    """(function, its tensors by name, library calls) for every operator; the tensors are made on the device index given."""
    def t(*shape, dtype=F32):
        return lambda index: _OnGpu(shape, dtype, index)

    rows, cols, units = 4, 64, 8
    mat, vec, row = t(rows, cols), t(cols), t(rows)
    opt = dict(post=vec, gate=t(2, cols), rng=t(2, dtype=I64))
    kw = lambda v: dict(post_weight=v["post"], gate=v["gate"], p=0.5, rng=v["rng"])  # noqa: E731
    x, w, y = t(rows, cols, dtype=BF), t(units, cols, dtype=BF), t(rows, units)
    return [
        (lambda v, **k: tw.dropout(v["x"], v["rng"], 0.5, out=v["out"], **k), dict(x=mat, out=mat, rng=opt["rng"])),
        (lambda v, **k: tw.join_rms_norm(v["r"], v["y"], v["w"], out=[v[n] for n in ("ro", "o", "q", "s", "rstd", "prstd")], **kw(v), **k),
         dict(r=mat, y=mat, w=vec, ro=mat, o=mat, q=t(rows, cols, dtype=U8), s=row, rstd=row, prstd=row, **opt)),
        (lambda v, **k: tw.join_rms_norm_bwd(v["g"], v["r"], v["rstd"], v["y"], v["w"], post_rstd=v["prstd"], d_residual=v["ds"],
                                             out=[v[n] for n in ("dr", "dy", "dw", "dp", "dg")], ws=v["ws"], **kw(v), **k),
         dict(g=mat, r=mat, rstd=row, y=mat, w=vec, prstd=row, ds=mat, dr=mat, dy=mat, dw=vec, dp=vec, dg=t(2, cols),
              ws=t(64, dtype=U8), **opt)),
        (lambda v, **k: tw.linear(v["x"], v["w"], v["b"], "relu", v["res"], out=v["y"], pre=v["pre"], ws=v["ws"], **k),
         dict(x=x, w=w, b=t(units), res=y, y=y, pre=t(rows, units, dtype=BF), ws=t(64, dtype=U8))),
        (lambda v, **k: tw.linear_bwd(v["g"], v["x"], v["w"], "relu", v["pre"], out=[v[n] for n in ("dx", "dw", "db")], ws=v["ws"], **k),
         dict(g=y, x=x, w=w, pre=t(rows, units, dtype=BF), dx=x, dw=w, db=t(units), ws=t(64, dtype=U8))),
    ]


@pytest.mark.parametrize("which", range(5))
def test_devices_and_streams(which, library):  # noqa: F811
    """Tensors of different devices and streams of another are refused; a call runs on the device of its tensors, whatever the
    current one."""
    call, tensors = _calls()[which]
    for index in (0, 1):
        call({n: make(index) for n, make in tensors.items()})
        assert library.calls[-1][1:] == (index, 1000 + index) and library.current == [0]
    call({n: make(1) for n, make in tensors.items()}, stream=_Stream(1))
    assert library.calls[-1][1:] == (1, 77)
    made = len(library.calls)
    for other in tensors:
        with pytest.raises(ValueError, match="must be on cuda:"):
            call({n: make(1 if n == other else 0) for n, make in tensors.items()})
    with pytest.raises(ValueError, match="stream"):
        call({n: make(1) for n, make in tensors.items()}, stream=_Stream(0))
    assert len(library.calls) == made


@pytest.mark.parametrize("which", range(5))
def test_shapes_and_types(which, library):  # noqa: F811
    """Every tensor of another shape, and those of fixed types of another type, are refused before the library is called."""
    call, tensors = _calls()[which]
    for other in tensors:
        if other == "ws":
            continue
        for wrong in (lambda o: _OnGpu(tuple(o.shape) + (1,), o.dtype), lambda o: _OnGpu(o.shape, torch.float16),
                      lambda o: _OnGpu(o.shape, o.dtype, contiguous=False)):
            v = {n: make(0) for n, make in tensors.items()}
            v[other] = wrong(v[other])
            with pytest.raises((ValueError, TypeError)):
                call(v)
    assert not library.calls


def test_dropout_needs_its_generator():
    from activation_sparse_ffn_03_amd import autograd
    for p in (0.0, 0.5):
        with pytest.raises(ValueError, match="rng"):
            autograd.dropout(torch.zeros(2, 8, requires_grad=True), None, p)


@pytest.mark.parametrize("grad", [True, False])
def test_nothing_is_kept_where_no_gradient_is_recorded(grad, monkeypatch):
    """Under no_grad the layers' parameters ask for a gradient all the same: the forward keeps no pre-activation, statistics
    or generator's state."""
    from activation_sparse_ffn_03_amd import autograd
    kept = []

    def linear(x, w, pre=None, **kw):
        kept.append(pre is not None)
        return torch.zeros(x.shape[0], w.shape[0], dtype=BF)

    def join(residual, y, weight, stats=False, **kw):
        kept.append(stats)
        rows = torch.zeros(residual.shape[0])
        return tw.JoinOut(residual.clone(), residual.clone(), None, None, rows, None)

    monkeypatch.setattr(tw, "linear", linear)
    monkeypatch.setattr(tw, "join_rms_norm", join)
    monkeypatch.setattr(tw, "dropout", lambda x, *a, **kw: x.clone())
    layer = autograd.TwellLinear(8, 16, act="silu", device="cpu")
    norm = autograd.TwellJoin(16, post_norm=False, dtype=F32, device="cpu")
    with torch.set_grad_enabled(grad):
        y = layer(torch.zeros(2, 3, 8, dtype=BF))
        r, out = norm(torch.zeros(2, 3, 16), y.float())
        d = autograd.dropout(layer.bias, tw.make_rng(1, device="cpu"), 0.5)
    assert kept == [grad, grad]
    assert all((t.grad_fn is not None) == grad for t in (y, r, out, d))
    assert y.shape == (2, 3, 16) and out.shape == (2, 3, 16) and d.shape == (16,)


def test_sizes_beyond_32_bits_are_refused(library):  # noqa: F811
    far = (1 << 32) + 64
    t = lambda *shape, dtype=F32: _OnGpu(shape, dtype)  # noqa: E731
    for call in (lambda: tw.dropout(t(2, far), t(2, dtype=I64), 0.5), lambda: tw.join_rms_norm(t(2, far), t(2, far), t(far)),
                 lambda: tw.join_rms_norm_bwd(t(2, far), t(2, far), t(2), t(2, far), t(far)),
                 lambda: tw.linear(t(2, far, dtype=BF), t(3, far, dtype=BF)), lambda: tw.linear(t(2, 64, dtype=BF), t(far, 64, dtype=BF)),
                 lambda: tw.linear_bwd(t(2, 3), t(2, far, dtype=BF), t(3, far, dtype=BF))):
        with pytest.raises(tw.TwellError, match="UNSUPPORTED"):
            call()
    assert not library.calls


# ---------------------------------------------------------------- kernels

@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    gxx, rocm = shutil.which("g++"), _rocm()
    if gxx is None or rocm is None:
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path_factory.mktemp("plans") / "linear_plan_print")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I",
                        os.path.join(ROOT, "include"), "-I", CSRC_OPS, "-I", CSRC,
                        os.path.join(ROOT, "tests", "linear_plan_print.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(layout, sizes):
        out = subprocess.run([exe], input="".join("%d %d %d %d\n" % (layout, *s) for s in sizes), capture_output=True, text=True)
        return [tuple(line.split()) for line in out.stdout.splitlines()]
    return ask


TILES = ("few", "mid", "wide", "big")


def test_every_product_is_reached(plans):
    for layout, sizes in ((0, variants.ROWS), (1, variants.OTHERS), (2, variants.COLS)):
        seen = set(plans(layout, sizes))
        want = {(t, s, k) for t in TILES for s in ("whole", "split") for k in ("aligned", "any")} - {("big", s, "any") for s in ("whole", "split")}
        want |= {("few", "whole", "copied"), ("big", "whole", "copied")}
        if layout == 2:
            want |= {("tall", "whole", "aligned"), ("tall", "split", "aligned")}
        assert want <= seen, (layout, want - seen)


def test_every_epilogue_is_reached(plans):
    seen = {(t, k) for t, _, k in plans(0, variants.EPILOGUES)}
    assert seen >= {(t, k) for t in TILES for k in ("aligned", "any")} - {("big", "any")}, seen


TILED = sorted(s for s in b.OPS_SOURCES if s.startswith(("linear_rows", "linear_mixed", "linear_cols", "linear_pair")))


@pytest.mark.parametrize("source", ["linear_rows_few.hip", "linear_mixed.hip", "linear_cols.hip", "linear_pair.hip"])
def test_waits_in_front_of_loads_into_lds(source):
    """As test_lds_load_wait_cpu.py, of which the tiles' header is the same in every source."""
    loads, m0, base = hazards(_listing(os.path.join(CSRC_OPS, source)))
    assert loads > 0 and not m0 and not base, (loads, len(m0), len(base))
    text = open(os.path.join(CSRC_OPS, "linear_tiled.h")).read()
    assert all("linear_tiled.h" in open(os.path.join(CSRC_OPS, s)).read() for s in TILED) and text.count("global_load_lds_dwordx4") == 2
