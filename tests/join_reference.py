"""The join of a block's output to the stream, its gradient and dropout's mask in float64 and whole numbers on the CPU, and
how far fp32 kernels may be from them."""
from __future__ import annotations

import numpy as np
import torch

from norm_reference import ROW_ADDS, U, half_step

M32 = (1 << 32) - 1


def philox(c, k):
    """The Philox4x32-10 block of counter words c and key words k (numbers or uint64 arrays)."""
    c, k = [np.asarray(v, dtype=np.uint64) for v in c], list(k)
    hi, lo = lambda v: v >> np.uint64(32), lambda v: v & np.uint64(M32)  # noqa: E731
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [hi(b) ^ c[1] ^ np.uint64(k[0]), lo(b), hi(a) ^ c[3] ^ np.uint64(k[1]), lo(a)]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def threshold(p: float) -> int:
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def kept(rows, cols, p, seed, step, site, first_row=0):
    """Which elements of rows first_row.. dropout keeps: bool [rows, cols]."""
    g = -(-cols // 8)
    full = lambda v: np.broadcast_to(np.asarray(v, dtype=np.uint64), (rows, g))  # noqa: E731
    words = philox([full(np.arange(g)[None, :]), full(np.arange(first_row, first_row + rows)[:, None]), full(step & M32),
                    full(site)], [seed & M32, seed >> 32 & M32])
    bits = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1).reshape(rows, -1)[:, :cols]
    return torch.from_numpy(bits.astype(np.int64) >= threshold(p))


def factor(p: float) -> float:
    """What dropout multiplies a kept element with, as the fp32 number it is."""
    d = threshold(p)
    return 0.0 if d == 65536 else float(np.float32(65536 / (65536 - d)))


def gate_rows(gate, rows):
    """The gate of every row, float64 [rows, cols] or 1."""
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    g = gate.double().reshape(-1, gate.shape[-1])
    return g.repeat_interleave(rows // g.shape[0], 0) if rows else g[:0]


def stream64(r, y, post, gate, alpha, eps, keep, p):
    """(r' in float64 before its rounding, rho_y or None)."""
    v, rho_y = y.double(), None
    if post is not None:
        rho_y = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
        v = v * rho_y * post.double()
    if keep is not None:
        v = torch.where(keep, v * factor(p), 0.0)
    return float(np.float32(alpha)) * r.double() + gate_rows(gate, y.shape[0]) * v, rho_y


def stream_tol(r, y, post, gate, alpha, eps, keep, p):
    """|r' - stream64|: rho_y is off as the norm's is ((ROW_ADDS + 1) / 2 roundings of the sum, mean, eps, root and
    quotient), y rho_y post_w and the factor add three, alpha r one, the last sum one; then the type's own."""
    want, rho_y = stream64(r, y, post, gate, alpha, eps, keep, p)
    ar = (float(np.float32(alpha)) * r.double()).abs()
    u = (want - float(np.float32(alpha)) * r.double()).abs()
    tol = u * ((((ROW_ADDS + 1) / 2 + 4 if post is not None else 0) + 3) * U) + ar * U + (want.abs() + u + ar) * U
    if r.dtype != torch.float32:
        tol = tol + half_step(r.dtype) * (want.abs() + tol)
    return tol


def backward64(d_out, d_res, r, rho, y, rho_y, w, post, gate, alpha, keep, p):
    """(dr, dy, dw, dpost, dgate) in float64; dgate [gate rows, cols]."""
    x, g, w, rho = r.double(), d_out.double(), w.double(), rho.double().reshape(-1, 1)
    rows, cols = x.shape
    xh, u = x * rho, g * w
    G = rho * (u - xh * (u * xh).mean(1, keepdim=True))
    if d_res is not None:
        G = G + d_res.double()
    m = torch.ones_like(x) if keep is None else torch.where(keep, factor(p), 0.0).double()
    gr = gate_rows(gate, rows)
    dv = G * m * gr
    dpost, dy, v = None, dv, y.double()
    if post is not None:
        ry = rho_y.double().reshape(-1, 1)
        yh = v * ry
        v = yh * post.double()
        t = dv * post.double()
        dy = ry * (t - yh * (t * yh).mean(1, keepdim=True))
        dpost = (dv * yh).sum(0)
    dgate = None
    if gate is not None:
        n = gate.reshape(-1, cols).shape[0]
        dgate = (G * torch.where(m > 0, m * v, 0.0)).reshape(n, rows // n, cols).sum(1)
    return float(np.float32(alpha)) * G, dy, (g * xh).sum(0), dpost, dgate


def backward_tol(d_out, d_res, r, rho, y, rho_y, w, post, gate, alpha, keep, p):
    """How far dr, dy, dw, dpost and dgate may be off. A row's sums are off by ROW_ADDS roundings of their absolute terms
    and those that a term has gathered; sums over rows are chains of at most rows / 256 + 1 of a thread, 32 rows side by
    side, 16 partial rows of a wave and 16 waves."""
    x, g, w, rho = r.double(), d_out.double(), w.double(), rho.double().reshape(-1, 1)
    rows, cols = x.shape
    xh, u = (x * rho).abs(), (g * w).abs()
    mean_abs = (u * xh).mean(1, keepdim=True)
    terms = rho * (u + xh * mean_abs)
    tG = terms * 6 * U + rho * xh * mean_abs * (ROW_ADDS + 3) * U
    base = rho * u
    if d_res is not None:
        tG = tG + 2 * U * (d_res.double().abs() + terms)
        base = base + d_res.double().abs()
    dr, dy, _, _, _ = backward64(d_out, d_res, r, rho, y, rho_y, w.float() if w.dtype == torch.float64 else w, post, gate, alpha, keep, p)
    al = abs(float(np.float32(alpha)))
    t_dr = al * tG + dr.abs() * U
    m = torch.ones_like(x) if keep is None else torch.where(keep, factor(p), 0.0).double()
    k = m * gate_rows(gate, rows).abs()
    big = terms if d_res is None else terms + d_res.double().abs()  # |G| and more
    t_dv = k * (tG + big * 3 * U)
    v = y.double().abs()
    t_dy, t_post = t_dv, None
    chain = (-(-rows // 256) + 1 + 32 + 16 + 16 + 3) * U
    if post is not None:
        ry, pw = rho_y.double().reshape(-1, 1), post.double().abs()
        yh = v * ry
        v = yh * pw
        kyh = k * v
        c1 = mean_abs
        err = (ROW_ADDS + 12) * U * (base * kyh).sum(1, keepdim=True) + \
            rho * c1 * (2 * ROW_ADDS + 16) * U * (xh * kyh).sum(1, keepdim=True)
        c2 = ((base * kyh).sum(1, keepdim=True) + rho * c1 * (xh * kyh).sum(1, keepdim=True)) / cols
        dv = k * big
        t_dy = ry * (pw * t_dv + dv * pw * 2 * U + yh * err / cols + yh * c2 * 4 * U) + 2 * U * ry * (dv * pw + yh * c2)
        t_post = ((t_dv + dv * 2 * U) * yh).sum(0) + (dv * yh).sum(0) * chain
    rounded = lambda t, val, like: t if like.dtype == torch.float32 else t + half_step(like.dtype) * (val.abs() + t)  # noqa: E731
    t_gate = None
    if gate is not None:
        n = gate.reshape(-1, cols).shape[0]
        fold = lambda a: a.reshape(n, rows // n, cols).sum(1)  # noqa: E731
        t_gate = fold(m * (tG + big * 5 * U) * v) + fold(m * big * v) * chain
    return rounded(t_dr, dr, r), rounded(t_dy, dy, y), (g * x * rho).abs().sum(0) * (chain + 2 * U), t_post, t_gate
