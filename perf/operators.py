"""Cases of the operators around the gate product: the residual-adding RMS norm with its E4M3 output and its gradient,
and the MX4 (blocks of 32 four-bit floats with one power-of-two scale) quantisation and product.

A case's "op" is one of

  norm       the residual's addition, the norm, and with codes the norm's E4M3 codes and row scales
  norm_grad  the norm's backward: gradients of the residual (and of what was added to it) and of the weight
  mx4_round  quantisation to MX4 and back, as quantisation-aware code sees a tensor
  mx4_linear a product with MX4 weights, the activations quantised within the call

Types are "bf16" or "f32"; "none" for an absent addition.
"""
import math

import torch

own = False
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "none": 0}


def listed():
    return [
        # one token of a 7B-class decode step: bf16 residual stream, the block's fp32 output added, codes for an FP8 gate
        dict(name="norm 1x4096 decode", op="norm", rows=1, cols=4096, res="bf16", delta="f32", out="bf16", codes=True),
        # a 1B-class batch whose residual stream is kept in fp32
        dict(name="norm 4096x2048 fp32 stream", op="norm", rows=4096, cols=2048, res="f32", delta="f32", out="bf16", codes=True),
        # a 7B-class prompt batch, an attention output in bf16 added
        dict(name="norm 16384x4096 prompt", op="norm", rows=16384, cols=4096, res="bf16", delta="bf16", out="bf16", codes=True),
        # the first norm of an fp32 network of odd width: nothing to add, no codes
        dict(name="norm 997x1999 odd fp32", op="norm", rows=997, cols=1999, res="f32", delta="none", out="f32", codes=False),
        # the training step: the block's fp32 input gradient comes back through the norm, joined by the stream's own
        dict(name="norm_grad 8192x2048 training", op="norm_grad", rows=8192, cols=2048, res="bf16", grad="f32", stream=True),
        # a small ragged fp32 batch, the last norm of a network: no gradient from the stream
        dict(name="norm_grad 131x1000 ragged", op="norm_grad", rows=131, cols=1000, res="f32", grad="f32", stream=False),
        # a 7B-class gate weight
        dict(name="mx4_round 11008x4096 weight", op="mx4_round", rows=11008, cols=4096, type="bf16"),
        # fp32 activations whose width leaves a part of a block
        dict(name="mx4_round 333x1990 ragged", op="mx4_round", rows=333, cols=1990, type="f32"),
        # one token against a 7B-class gate weight
        dict(name="mx4_linear 1x4096x11008 decode", op="mx4_linear", rows=1, cols=4096, units=11008, x="bf16", y="bf16"),
        # a small decode batch, 1B-class
        dict(name="mx4_linear 24x2048x5632 decode", op="mx4_linear", rows=24, cols=2048, units=5632, x="bf16", y="f32"),
        # nothing a multiple of a tile
        dict(name="mx4_linear 1003x1990x8100 odd", op="mx4_linear", rows=1003, cols=1990, units=8100, x="f32", y="f32"),
        # a 7B-class prompt batch
        dict(name="mx4_linear 16384x4096x11008", op="mx4_linear", rows=16384, cols=4096, units=11008, x="bf16", y="bf16"),
    ]


def draw(rng):
    def spread(lo, hi, step):
        n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        n = int(round(n)) if rng.random() < 0.4 else int(round(n / step)) * step
        n = min(max(n, lo), hi)
        return n if n != 3072 else n + step

    op = rng.choice(["norm", "norm", "norm_grad", "mx4_round", "mx4_linear", "mx4_linear"])
    any_type = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    cols = spread(64, 8192, 64)
    if op == "norm":
        c = dict(op=op, rows=spread(1, 16384, 16), cols=cols, res=any_type(), delta=rng.choice(["bf16", "f32", "none"]),
                 out=any_type(), codes=rng.random() < 0.6)
    elif op == "norm_grad":
        c = dict(op=op, rows=spread(1, 8192, 16), cols=cols, res=any_type(), grad=any_type(), stream=rng.random() < 0.7)
    elif op == "mx4_round":
        c = dict(op=op, rows=spread(1, 11008, 16), cols=cols, type=any_type())
    else:
        c = dict(op=op, rows=spread(1, 16384, 16), cols=cols, units=spread(256, 14336, 64), x=any_type(), y=any_type())
    top = [work(d) for d in listed() if d["op"] == op]
    while any(work(c)[k] > max(t[k] for t in top) for k in ("bytes", "flops")):
        c["rows"] = c["rows"] * 3 // 4
    return c


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _stream(gen, rows, cols, dtype):
    """A residual stream: rows of different size, a few channels that stand out in all of them, padding rows of zeros."""
    dev = gen.device
    v = torch.randn(rows, cols, generator=gen, device=dev)
    v *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=dev))
    v[:, torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device=dev)] *= 20
    v[torch.arange(rows, device=dev) % 64 == 37] = 0
    return v.to(dtype)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, cols = case["rows"], case["cols"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=dev)

    s = dict(case)
    if case["op"] == "norm":
        res, out = TYPES[case["res"]], TYPES[case["out"]]
        s["residual"] = _stream(gen, rows, cols, res)
        s["delta"] = None
        if case["delta"] != "none":
            s["delta"] = (0.3 * randn(rows, cols)).to(TYPES[case["delta"]])
            s["delta"][torch.arange(rows, device=dev) % 64 == 37] = 0
        s["weight"] = (1 + 0.2 * randn(cols)).to(out)
        # what a serving program keeps: the new residual, the norm, its codes, their scales, no saved statistics
        q = case["codes"]
        s["buffers"] = (empty(rows, cols, dtype=res), empty(rows, cols, dtype=out),
                        empty(rows, cols, dtype=torch.uint8) if q else None, empty(rows, dtype=torch.float32) if q else None, None)
    elif case["op"] == "norm_grad":
        res = TYPES[case["res"]]
        s["residual"] = _stream(gen, rows, cols, res)
        s["weight"] = (1 + 0.2 * randn(cols)).to(res)
        s["rstd"] = (s["residual"].float().square().mean(1) + EPS).rsqrt()
        s["d_out"] = (0.01 * randn(rows, cols)).to(TYPES[case["grad"]])
        s["d_residual"] = (0.01 * randn(rows, cols)).to(res) if case["stream"] else None
    elif case["op"] == "mx4_round":
        s["value"] = _stream(gen, rows, cols, TYPES[case["type"]])
    else:
        units = case["units"]
        s["value"] = _stream(gen, rows, cols, TYPES[case["x"]])
        w = randn(units, cols) / math.sqrt(cols)
        s["codes"], s["scales"] = _pack(*_quantize(w))
        s["out"] = empty(rows, units, dtype=TYPES[case["y"]])
    return s


# The plain forms.


def _quantize(v):
    """fp32 [rows, cols] to the E2M1 values it rounds to ([rows, blocks, 32], zeros behind the last column) and scale codes [rows, blocks]."""
    rows, cols = v.shape
    blocks = -(-cols // 32)
    v = torch.nn.functional.pad(v, (0, 32 * blocks - cols)).view(rows, blocks, 32)
    big = v.abs().amax(2)
    code = ((big.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = v.abs() * ((254 - code) << 23).view(torch.float32)[:, :, None]  # exact: over a power of two
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6), v)  # round() takes ties to even
    bad = ~torch.isfinite(big)
    return torch.where(bad[:, :, None], torch.zeros_like(q), q), torch.where(bad, 255, code)


def _pack(q, code):
    """Values and scale codes to bytes: two codes a byte, the even column's in the low half; rows filled with zeros to whole
    128 columns of codes (64 bytes) and whole 512 columns of scales (16 bytes)."""
    a = q.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    c = c.view(c.shape[0], -1, 2)
    c = c[:, :, 0] | (c[:, :, 1] << 4)
    pad = torch.nn.functional.pad
    return pad(c, (0, -c.shape[1] % 64)).contiguous(), pad(code.to(torch.uint8), (0, -code.shape[1] % 16)).contiguous()


def _unpack(codes):
    """Bytes to the E2M1 values [rows, blocks, 32]."""
    c = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1, 32)
    m = (c & 7).float()
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c > 7, -a, a)


def _scaled(q, code, cols):
    """Values times their scales, fp32 [rows, cols]."""
    code = code[:, :q.shape[1], None].to(torch.int32)
    s = torch.where(code == 0, 1 << 22, code << 23).view(torch.float32)
    s = torch.where(code == 255, math.nan, s)
    return (q * s).view(q.shape[0], -1)[:, :cols]


def _norm(s):
    r = s["residual"].float()
    if s["delta"] is not None:
        r = r + s["delta"].float()
    r = r.to(s["residual"].dtype)
    x = r.float()
    n = x * (1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)) * s["weight"].float()
    got = [r, n.to(TYPES[s["out"]])]
    if s["codes"]:
        scale = n.abs().amax(1) / 448
        scale = torch.where(scale > 0, scale, 1.0)
        got += [(n / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale]
    return got


def _norm_grad(s):
    g, w = s["d_out"].float(), s["weight"].float()
    hat = s["residual"].float() * s["rstd"][:, None]
    u = g * w
    dr = (u - hat * (u * hat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["d_residual"] is not None:
        dr = dr + s["d_residual"].float()
    return [dr.to(s["residual"].dtype), (g * hat).sum(0)]


def _mx4_round(s):
    q, code = _quantize(s["value"].float())
    return [_scaled(q, code, s["cols"]).to(s["value"].dtype), code.to(torch.uint8)]


def _mx4_linear(s):
    x = _scaled(*_quantize(s["value"].float()), s["cols"])
    w = _scaled(_unpack(s["codes"]), s["scales"], s["cols"])
    return [torch.matmul(x, w.t()).to(TYPES[s["y"]])]


def run(s):
    if not own:
        return {"norm": _norm, "norm_grad": _norm_grad, "mx4_round": _mx4_round, "mx4_linear": _mx4_linear}[s["op"]](s)
    from activation_sparse_ffn_03_amd import twell as tw
    if s["op"] == "norm":
        got = tw.add_rms_norm(s["residual"], s["weight"], delta=s["delta"], eps=EPS, out=s["buffers"])
        return [got.residual, got.out] + ([got.codes.view(torch.float8_e4m3fn), got.scale] if s["codes"] else [])
    if s["op"] == "norm_grad":
        return list(tw.add_rms_norm_bwd(s["d_out"], s["residual"], s["rstd"], s["weight"], d_residual=s["d_residual"]))
    if s["op"] == "mx4_round":
        codes, scales = tw.quantize_mx4(s["value"])
        return [tw.dequantize_mx4(codes, scales, s["cols"], dtype=s["value"].dtype), scales[:, :-(-s["cols"] // 32)]]
    return [tw.linear_mx4(s["value"], s["codes"], s["scales"], out=s["out"])]


def work(case):
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    blocks = -(-cols // 32)
    if case["op"] == "norm":
        b = n * (2 * SIZE[case["res"]] + SIZE[case["delta"]] + SIZE[case["out"]]) + cols * SIZE[case["out"]]
        return {"bytes": b + ((n + 4 * rows) if case["codes"] else 0), "flops": 7 * n}
    if case["op"] == "norm_grad":
        b = n * (SIZE[case["res"]] * (3 if case["stream"] else 2) + SIZE[case["grad"]]) + 4 * rows + cols * (SIZE[case["res"]] + 4)
        return {"bytes": b, "flops": 10 * n}
    if case["op"] == "mx4_round":
        return {"bytes": 2 * n * SIZE[case["type"]] + 2 * rows * blocks * 17, "flops": 4 * n}
    b = n * SIZE[case["x"]] + case["units"] * blocks * 17 + rows * case["units"] * SIZE[case["y"]]
    return {"bytes": b, "flops": 2 * n * case["units"]}


# The definitions in 64 bits.

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(e):
    """2^e in float64 for whole e, by its bits: a library's power may be a last place off, and a value half way between two levels shows it."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx4(v):
    """The value each element of a finite float64 [rows, cols] stands for after quantisation, and the exponents of the blocks."""
    rows, cols = v.shape
    blocks = -(-cols // 32)
    full = v.new_zeros(rows, 32 * blocks)
    full[:, :cols] = v
    full = full.view(rows, blocks, 32)
    big = full.abs().max(2).values
    e = (torch.frexp(big).exponent - 3).clamp(min=-127)  # big = m * 2^k with m in [1/2, 1): floor(log2) - 2 is k - 3
    e = torch.where(big > 0, e, -127)
    unit = _power(e)[:, :, None]
    a = full.abs() / unit
    k = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):  # half way between two levels goes to the one with the even number
        mid = (_LEVELS[i] + _LEVELS[i + 1]) / 2
        k += (a > mid) if i % 2 == 0 else (a >= mid)
    q = torch.tensor(_LEVELS, dtype=v.dtype, device=v.device)[k] * torch.sign(full) * unit
    return q.view(rows, -1)[:, :cols], e


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["residual"].double()
        if s["delta"] is not None:
            r = r + s["delta"].double()
        r = r.to(s["residual"].dtype).double()  # the norm is that of the residual as stored
        n = r / ((r ** 2).sum(1) / case["cols"] + EPS).sqrt()[:, None] * s["weight"].double()
        got = [r, n]
        if case["codes"]:
            top = n.abs().max(1).values
            top = torch.where(top > 0, top / 448, torch.ones_like(top))
            got += [n / top[:, None], top]
        return got
    if case["op"] == "norm_grad":
        # with y = w x / |x|_eps: the part of u along x is taken out of u / |x|_eps
        x, rho = s["residual"].double(), s["rstd"].double()[:, None]
        u = s["d_out"].double() * s["weight"].double()
        dr = rho * u - rho ** 3 * x * (u * x).sum(1, keepdim=True) / case["cols"]
        if case["stream"]:
            dr += s["d_residual"].double()
        return [dr, torch.sum(s["d_out"].double() * x * rho, 0)]
    if case["op"] == "mx4_round":
        q, e = _exact_mx4(s["value"].double())
        return [q, (e + 127).to(torch.uint8)]
    x, _ = _exact_mx4(s["value"].double())
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).flatten(1)[:, :case["cols"]].long()
    w = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float64, device=c.device)[c]
    w *= _power(s["scales"].long() - 127).repeat_interleave(32, 1)[:, :case["cols"]]
    return [x @ w.T]
