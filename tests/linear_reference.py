"""The linear layer and its gradients in float64, and how far fp32 kernels of bf16 operands may be from them."""
from __future__ import annotations

import math

import torch

from norm_reference import U, half_step

CDF = 7.5e-8  # what formula 26.2.17 of Abramowitz and Stegun may be off by


def cdf(z):
    return torch.special.ndtr(z)


def density(z):
    return torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * cdf(z)}[act]()


def slope64(z, act):
    s = torch.sigmoid(z)
    return {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(), "silu": lambda: s * (1 + z * (1 - s)),
            "gelu": lambda: cdf(z) + z * density(z)}[act]()


def act_tol(z, act):
    """The exponential is off by 2 |z| + 2 roundings (its argument's product and constant, its own last place), what it goes
    through by at most 6 more; below exp's range SiLU gives 0. GELU: the formula's error and at most 12 roundings."""
    if act == "silu":
        return (z * torch.sigmoid(z)).abs() * (2 * z.abs() + 6) * U + 1e-36
    if act == "gelu":
        return z.abs() * (CDF + 12 * U)
    return torch.zeros_like(z)


def slope_tol(z, act):
    if act == "silu":
        return torch.sigmoid(z) * (1 + z.abs()) * (2 * z.abs() + 8) * U + 1e-36
    if act == "gelu":
        return CDF + 12 * U + z.abs() * density(z) * (z * z + 8) * U
    return torch.zeros_like(z)


def rounded(tol, value, dtype):
    return tol if dtype == torch.float32 else tol + half_step(dtype) * (value.abs() + tol)


def forward(x, w, bias, act, residual, dtype):
    """((z, its bound before rounding), (y, its bound)): a sum of k exact products has at most k roundings of the sum of their
    magnitudes, whatever the order."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    tol = (x.abs() @ w.abs().t()) * x.shape[1] * U
    if bias is not None:
        z = z + bias.double()
        tol = tol + (z.abs() + tol) * U
    y, ty = act64(z, act), 1.13 * tol + act_tol(z, act)  # no slope above 1.13
    if residual is not None:
        y = y + residual.double()
        ty = ty + (y.abs() + ty) * U
    return (z, tol), (y, rounded(ty, y, dtype))


def backward(d_out, x, w, act, pre, dx_dtype, dw_dtype):
    """((dx, bound), (dw, bound), (db, bound))."""
    g, x, w = d_out.double(), x.double(), w.double()
    dz, t = g, torch.zeros_like(g)
    if act != "none":
        z = pre.double()
        dz = g * slope64(z, act)
        t = g.abs() * slope_tol(z, act) + dz.abs() * U
    rows = g.shape[0]
    db = (dz.sum(0), (t + dz.abs() * (-(-rows // 256) + 72) * U).sum(0))
    if act != "none" or d_out.dtype != torch.bfloat16:
        t = t + half_step(torch.bfloat16) * (dz.abs() + t)
    size = dz.abs() + t
    dx, dw = dz @ w, dz.t() @ x
    tx = t @ w.abs() + (size @ w.abs()) * w.shape[0] * U
    tw = t.t() @ x.abs() + (size.t() @ x.abs()) * rows * U
    return (dx, rounded(tx, dx, dx_dtype)), (dw, rounded(tw, dw, dw_dtype)), db
