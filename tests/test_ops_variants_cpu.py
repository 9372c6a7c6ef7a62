"""Every kernel variant that a call of the operators around the block can reach is reached by a size of the GPU tests:
the plans are asked of the library's own header, on the CPU."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

import test_gpu_mx4 as mx4
import test_gpu_norm as norm
import test_gpu_ops_variants as more
from test_host_sanitize import CSRC, ROOT, _rocm

CSRC_OPS = os.path.join(ROOT, "activation_sparse_ffn_03_amd", "csrc_ops")


def _sizes(test, names):
    """Argument tuples of the parametrize mark of a test that names them."""
    marks = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names]
    assert len(marks) == 1
    return list(marks[0].args[1])


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    gxx, rocm = shutil.which("g++"), _rocm()
    if gxx is None or rocm is None:
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path_factory.mktemp("plans") / "mx4_plan_print")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I",
                        os.path.join(ROOT, "include"), "-I", CSRC_OPS, "-I", CSRC,
                        os.path.join(ROOT, "tests", "mx4_plan_print.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(sizes):
        out = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in sizes), capture_output=True, text=True)
        return [line.split() for line in out.stdout.splitlines()]
    return ask


def _variant(plan, n, cols, x, f):
    """What launch_mx4_product instantiates."""
    if plan == "fused":
        return plan, x, "1x1" if n <= 4 else "2x1" if n <= 16 else "2x2", "tail" if cols % 8 else "whole"
    if plan == "direct":
        return plan, f
    half = "half" if -(-cols // 128) % 2 else "whole"
    return plan, half, "one" if cols <= 256 else "many", "few" if n < 128 else "full"


EVERY_PRODUCT = ({("fused", x, t, w) for x in ("bf16", "f32") for t in ("1x1", "2x1", "2x2") for w in ("tail", "whole")} |
                 {("direct", f) for f in "124"} |
                 {(p, h, o, "full") for p in ("mid", "big") for h in ("half", "whole") for o in ("one", "many")} |
                 {("mid", h, "many", "few") for h in ("half", "whole")})


def test_every_product_variant_is_reached(plans):
    names = "n,cols,units"
    both = mx4.PRODUCTS + _sizes(mx4.test_large_products_are_exact, names) + more.EXACT
    single = _sizes(mx4.test_large_products, names)
    seen = set()
    for sizes, types in ((both, ("bf16", "f32")), (single, ("f32",))):
        for (n, cols, units), (linear, matmul, f) in zip(sizes, plans(sizes)):
            for x in types:
                seen.add(_variant(linear, n, cols, x, f))
            if sizes is not both or (n, cols, units) in mx4.PRODUCTS:
                seen.add(_variant(matmul, n, cols, None, f))
    assert seen == EVERY_PRODUCT, (EVERY_PRODUCT - seen, seen - EVERY_PRODUCT)


def test_nan_blocks_meet_every_kind_of_product(plans):
    sizes = [(n, cols, units) for n, units in _sizes(mx4.test_nan_blocks_mark_their_row_and_column, "n,units")
             for cols in _sizes(mx4.test_nan_blocks_mark_their_row_and_column, "cols")] + more.NAN
    seen = {(linear, n < 128) if linear == "mid" else linear for (n, _, _), (linear, _, _) in zip(sizes, plans(sizes))}
    assert seen == {"fused", "direct", ("mid", False), ("mid", True), "big"}


def test_scale_ranges_meet_every_kind_of_product(plans):
    seen = {(matmul, n < 128) if matmul == "mid" else (matmul, f) if matmul == "direct" else matmul
            for (n, _, _), (_, matmul, f) in zip(more.RANGE, plans(more.RANGE))}
    assert seen == {("direct", f) for f in "124"} | {("mid", False), ("mid", True), "big"}


# widths at which the norm and its backward change their number of threads or chunks a thread
STEPS = [128, 256, 512, 1024, 2048, 4096, 8192, 16384]


def _norm_variants(widths):
    return {(next(s for s in STEPS if w <= s), "short" if w < 8 else "any" if w % 8 else "aligned") for w in widths}


EVERY_NORM = {(s, k) for s in STEPS for k in ("any", "aligned")} | {(128, "short")}


def test_every_norm_variant_is_reached():
    assert _norm_variants(norm.WIDTHS + more.NORM_WIDTHS) == EVERY_NORM
    assert _norm_variants([c for _, c in _sizes(norm.test_backward, "rows,cols") + more.BACKWARD]) == EVERY_NORM
