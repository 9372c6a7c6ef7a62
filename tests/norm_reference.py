"""The norm, its gradient and E4M3 codes in float64 on the CPU, and how far fp32 kernels may be from them."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32, relative
# Additions one thread makes in a row's sum (at most 64 elements), the wave's six steps and the workgroup's four.
ROW_ADDS = 64 + 6 + 4


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def forward64(residual, delta, weight, eps):
    """(r' in the residual's dtype, n, rho): r' is the fp32 sum rounded once to the residual's dtype."""
    r = residual if delta is None else (residual.float() + delta.float()).to(residual.dtype)
    x = r.double()
    rho = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    return r, x * rho * weight.double(), rho


def forward_tol(n, dtype):
    """|out - n|: the sum of squares is off by ROW_ADDS + 1 roundings of positive terms, which the root halves; the
    mean, eps, the root, the quotient and the two products add one each; then the output's own rounding."""
    rel = ((ROW_ADDS + 1) / 2 + 6) * U
    return n.abs() * (rel + (0 if dtype == torch.float32 else half_step(dtype) * (1 + rel)))


def backward64(d_out, d_residual, r, rho, weight):
    x, g, w = r.double(), d_out.double(), weight.double()
    rho = rho.double().reshape(-1, 1)
    xh, u = x * rho, g * w
    dr = rho * (u - xh * (u * xh).mean(1, keepdim=True))
    if d_residual is not None:
        dr = dr + d_residual.double()
    return dr, (g * xh).sum(0)


def backward_tol(d_out, d_residual, r, rho, weight, groups):
    """|dr - dr64| and |dw - dw64|. The row's mean is off by ROW_ADDS + 3 roundings of its absolute terms; what it
    meets in dr has at most 6 more. dw is a chain over one thread's rows and the rows side by side, then groups / 16 and 16 sums."""
    x, g, w = r.double(), d_out.double(), weight.double()
    rho = rho.double().reshape(-1, 1)
    xh, u = x * rho, g * w
    mean_abs = (u * xh).abs().mean(1, keepdim=True)
    terms = rho * (u.abs() + xh.abs() * mean_abs)
    tol = terms * 6 * U + rho * xh.abs() * mean_abs * (ROW_ADDS + 3) * U
    if d_residual is not None:
        tol = tol + 2 * U * (d_residual.double().abs() + terms)
    dr, _ = backward64(d_out, d_residual, r, rho, weight)
    if r.dtype != torch.float32:
        tol = tol + half_step(r.dtype) * (dr.abs() + tol)
    rows = r.shape[0]
    chain = -(-rows // groups) + 4 + -(-groups // 16) + 16 + 2
    return tol, (g * xh).abs().sum(0) * chain * U


def e4m3_values():
    """Value of every E4M3 code, NaN for 0x7F and 0xFF."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def e4m3_tol(v):
    """Half a step of the E4M3 grid at v (|v| <= 448): 2^-4 of the value, or half of the subnormals' 2^-9."""
    return torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
