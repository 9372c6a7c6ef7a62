"""Loads straight into LDS take their address from M0, and one wait state has to pass between a scalar write of M0 and
such a load (CDNA ISA, "required user-inserted wait states"); the same holds with five between a vector instruction's
write of a scalar register and a memory instruction that reads it. The compiler keeps both for its own instructions but
does not look into inline assembly: the listings of the kernels built here are checked, on the CPU."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from activation_sparse_ffn_03_amd import build as b


def _regs(operand: str) -> set:
    """Scalar registers of an operand."""
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.match(r"(s\d+|m0)$", operand) else set()


def hazards(listing: str):
    """(loads into LDS, those too close behind a write of M0, those too close behind a vector write of their base)."""
    seen, loads, m0, base = [], 0, [], []
    for line in listing.splitlines():
        line = line.split(";")[0].strip()
        if re.match(r"^[._A-Za-z$]\S*:", line):
            seen.append(("label", []))
            continue
        if not line or line.startswith("."):
            continue
        name, _, rest = line.partition(" ")
        operands = re.split(r"[,\s]+", rest.strip()) if rest else []
        if re.match(r"(global|buffer|scratch)_load_lds", name) or (name.startswith("buffer_load") and "lds" in operands):
            loads += 1
            read, passed = set().union(*map(_regs, operands)), 0
            for before, ops in reversed(seen[-8:]):
                if before == "label" or passed >= 5:
                    break
                written = _regs(ops[0]) if ops else set()
                if "m0" in written and passed < 1:
                    m0.append(line)
                if before.startswith("v_") and written & read:
                    base.append(line)
                passed += 1 + int(ops[0]) if before == "s_nop" else 1
        seen.append((name, operands))
    return loads, m0, base


def test_checker():
    load = "\tglobal_load_lds_dwordx4 v1, s[2:3]\n"
    assert hazards("\ts_mov_b32 m0, s1\n" + load)[:2] == (1, [load.strip()])
    assert hazards("\ts_mov_b32 m0, s1\n\ts_nop 0\n" + load) == (1, [], [])
    assert hazards("\ts_add_i32 m0, s1, s2\n\tv_mov_b32_e32 v2, 0\n" + load) == (1, [], [])
    assert hazards("\tv_readfirstlane_b32 s3, v0\n\ts_nop 3\n" + load)[2] == [load.strip()]
    assert hazards("\tv_readfirstlane_b32 s3, v0\n\ts_nop 4\n" + load) == (1, [], [])


def _listing(path: str) -> str:
    try:
        hipcc = b._hipcc()
    except Exception:
        pytest.skip("needs hipcc")
    flags = [f for f in b.HIP_FLAGS if f != "-Wall"]
    r = subprocess.run([hipcc, *flags, "-w", "-S", "--cuda-device-only", path, "-o", "-"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


@pytest.mark.parametrize("source", ["mx4_product.hip"])
def test_operators(source):
    loads, m0, base = hazards(_listing(os.path.join(b.CSRC_OPS, source)))
    assert loads > 0 and not m0 and not base, (loads, len(m0), len(base))


@pytest.mark.parametrize("source", ["gate_pack.hip", "up_blocked.hip", "bwd_blocked.hip"])
def test_block(source):
    loads, m0, base = hazards(_listing(os.path.join(b.CSRC, source)))
    assert loads > 0 and not m0 and not base, (loads, len(m0), len(base))


def test_backward_uses_none_of_its_header():
    assert hazards(_listing(os.path.join(b.CSRC, "bwd.hip")))[0] == 0


def test_every_source_with_such_loads_is_listed():
    """Sources that reach the statement, directly or through a header."""
    def reaches(path):
        text = open(path).read()
        if re.search(r"\bdma_16B\(", text.split("dma_16B(const void", 1)[-1] if path.endswith("twell_device.h") else text):
            return True
        return any(reaches(h) for inc in re.findall(r'#include "([^"]+)"', text)
                   if os.path.exists(h := os.path.join(os.path.dirname(path), inc)) and not h.endswith("twell_device.h"))

    found = {s for d, names in ((b.CSRC, b.SOURCES), (b.CSRC_OPS, b.OPS_SOURCES)) for s in names
             if reaches(os.path.join(d, s))}
    assert found == {"mx4_product.hip", "gate_pack.hip", "up_blocked.hip", "bwd_blocked.hip", "bwd.hip"}
