"""The operators around an optimizer step, as cases with inputs, a plain form and the framework's calls.

What comes in before the step: the gradients of many tensors, whose global norm is formed ("norm") and which
are clipped to it ("clip").  What goes out after it, or is kept from the forward pass for the Newton
preconditioner: matrices in microscaled 4-bit floating point, made from weights, activations and layer inputs
("quantize"), multiplied ("product") or multiplied with themselves ("gram").

4-bit values are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  Format "mx": one power-of-two scale
(E8M0) per 32 values, two below that of the largest.  Format "nv": one E4M3 scale per 16 values, a sixth of the largest,
and one fp32 scale per matrix, the smallest power of two that keeps the others within E4M3's 448.  Rounding is to
the nearest value, ties to the even code, in the codes and in the E4M3 scales.
"""
from __future__ import annotations

import math
import random

import torch

own = False

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mx": 32, "nv": 16}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}

# hidden 2048, 16 query and 8 key/value heads of 128, a gated MLP of 6144
LAYER = ((2048, 2048), (1024, 2048), (1024, 2048), (2048, 2048), (6144, 2048), (6144, 2048), (2048, 6144))


def listed():
    return [
        # the normalisation gains of a 28-layer model: 112 short fp32 vectors, each with its own norm too
        {"name": "norm of gains", "op": "norm", "set": "gains", "count": 28, "dtype": "f32", "each": True, "mix": 0},
        # every matrix gradient of a 1.4B-parameter model before the step
        {"name": "norm of a model", "op": "norm", "set": "layers", "count": 28, "dtype": "bf16", "each": False, "mix": 0},
        # a flat buffer of odd-sized tensors, some of them column slices
        {"name": "clip ragged", "op": "clip", "set": "ragged", "count": 40, "dtype": "f32", "out": "f32", "mix": 1},
        # gradients accumulated in fp32, handed to the step in bf16
        {"name": "clip accumulated", "op": "clip", "set": "layers", "count": 4, "dtype": "f32", "out": "bf16", "mix": 0},
        # the weights of one layer after the step, for the next forward pass
        {"name": "quantize mx weights", "op": "quantize", "rows": 6144, "cols": 2048, "count": 4, "dtype": "bf16", "format": "mx", "transpose": False},
        # a layer's input, tokens x features, kept feature by feature for the preconditioner
        {"name": "quantize nv input", "op": "quantize", "rows": 8192, "cols": 2048, "count": 1, "dtype": "bf16", "format": "nv", "transpose": True},
        # a small matrix of odd sizes
        {"name": "quantize mx ragged", "op": "quantize", "rows": 777, "cols": 333, "count": 1, "dtype": "f32", "format": "mx", "transpose": True},
        # one token through a projection
        {"name": "product one token", "op": "product", "m": 1, "n": 6144, "k": 2048, "format": "nv", "out": "bf16"},
        # a batch of odd sizes
        {"name": "product ragged", "op": "product", "m": 1000, "n": 777, "k": 1333, "format": "mx", "out": "f32"},
        # a training batch through a projection
        {"name": "product batch", "op": "product", "m": 8192, "n": 6144, "k": 2048, "format": "nv", "out": "bf16"},
        # one narrow layer's input over a short batch
        {"name": "gram of an input", "op": "gram", "d": 768, "tokens": 1000, "count": 1, "format": "nv"},
        # the layer inputs of four layers for the preconditioner
        {"name": "gram of inputs", "op": "gram", "d": 2048, "tokens": 8192, "count": 4, "format": "mx"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "clip", "quantize", "product", "product", "gram"))
    if op in ("norm", "clip"):
        kind = rng.choice(("gains", "layers", "ragged", "ragged"))
        most = {"gains": 28, "layers": 28 if op == "norm" else 4, "ragged": 300}[kind]
        case = {"op": op, "set": kind, "count": _log(rng, 1, most), "dtype": rng.choice(("bf16", "f32")), "mix": rng.randrange(1 << 20)}
        if op == "norm":
            case["each"] = kind != "layers" and rng.random() < 0.5
            if kind == "layers" and case["dtype"] == "f32":
                case["count"] = min(case["count"], 14)
        else:
            case["out"] = rng.choice(("bf16", "f32")) if case["dtype"] == "f32" else "bf16"
        return case
    fmt = rng.choice(("mx", "nv"))
    if op == "quantize":
        rows, cols = _log(rng, 1, 8192), _log(rng, 1, 8192)
        count = max(1, min(rng.randint(1, 6), (48 << 20) // (rows * cols)))
        return {"op": op, "rows": rows, "cols": cols, "count": count, "dtype": rng.choice(("bf16", "f32")), "format": fmt, "transpose": rng.random() < 0.5}
    if op == "product":
        n, k = _log(rng, 16, 8192), _log(rng, 16, 8192)
        m = _log(rng, 1, max(1, min(8192, 8192 * 6144 * 2048 // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "format": fmt, "out": rng.choice(("bf16", "f32"))}
    return {"op": op, "d": _log(rng, 64, 2048), "tokens": _log(rng, 64, 8192), "count": rng.randint(1, 4), "format": fmt}


# ------------------------------------------------------------------------------- inputs


def _shapes(case):
    """(rows, cols, leading dimension) of each tensor of a set, in the order of the flat buffer."""
    if case["set"] == "gains":
        return [(1, c, c) for c in (2048, 2048, 128, 128)] * case["count"]
    if case["set"] == "layers":
        return [(r, c, c) for r, c in LAYER] * case["count"]
    rng, out = random.Random(case["mix"]), []
    for _ in range(case["count"]):
        if rng.random() < 0.4:
            out.append((1, _log(rng, 1, 20000), 0))
        else:
            r, c = _log(rng, 1, 700), _log(rng, 1, 700)
            out.append((r, c, c + (rng.randint(1, 40) if rng.random() < 0.3 else 0)))
    return [(r, c, max(c, ld)) for r, c, ld in out]


def _views(flat, shapes):
    got, at = [], 0
    for r, c, ld in shapes:
        got.append(flat[at:at + r * ld].view(r, ld)[:, :c])
        at += r * ld
    return got


def _codes(index, sign, cols):
    """4-bit codes packed two to a byte (the even column in the low half), rows padded to 128 columns."""
    code = (index + 8 * sign).to(torch.uint8)
    code = torch.nn.functional.pad(code, (0, -cols % 128))
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _tiles(scales, rows, cols, block):
    """Scale bytes in tiles of 128 rows x 4 scales: byte 16 (r mod 32) + 4 (r div 32) + s of its tile; tiles row by row."""
    wide = -(-cols // 128) * 128 // block
    s = torch.nn.functional.pad(scales, (0, wide - scales.shape[1], 0, -rows % 128))
    return s.view(-1, 4, 32, wide // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _operand(gen, rows, cols, fmt, spread):
    """A matrix in 4-bit form, as the quantization leaves it: rows of their own size, normal values."""
    dev = torch.device("cuda")
    x = torch.randn(rows, cols, generator=gen, device=dev)
    if spread:
        x *= torch.exp(torch.rand(rows, 1, generator=gen, device=dev) * math.log(100.0) + math.log(0.1))
    index, sign, scales, whole = _plain_quantize(x.to(torch.bfloat16).float(), fmt)
    raw = (scales.to(torch.int32) + 127).to(torch.uint8) if fmt == "mx" else scales.to(torch.float8_e4m3fn).view(torch.uint8)
    return {"rows": rows, "cols": cols, "codes": _codes(index, sign, cols), "scales": _tiles(raw, rows, cols, BLOCK[fmt]), "whole": whole.reshape(1)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if own:
        import newton_schulz_hyperball_b200 as nshb
    if op in ("norm", "clip"):
        shapes = _shapes(case)
        flat = torch.randn(sum(r * ld for r, _, ld in shapes), generator=gen, device=dev)
        size = torch.exp(torch.rand(len(shapes), generator=gen, device=dev) * math.log(100.0) + math.log(1e-4))
        for i, v in enumerate(_views(flat, shapes)):
            v *= size[i]
        s["flat"] = flat.to(DTYPE[case["dtype"]])
        s["total"] = torch.zeros(2, device=dev)
        s["max_norm"] = 1.0 if op == "norm" else 0.25 * float(flat.norm())
        if any(c < ld for _, c, ld in shapes):
            # the places of the flat buffer that belong to a tensor
            s["at"] = torch.nonzero(torch.cat([(torch.arange(r * ld, device=dev) % ld) < c for r, c, ld in shapes])).reshape(-1)
        if op == "clip":
            s["out"] = torch.zeros(flat.numel(), dtype=DTYPE[case["out"]], device=dev)
        elif case["each"]:
            s["each"] = torch.zeros(len(shapes), device=dev)
            s["owner"] = torch.repeat_interleave(torch.arange(len(shapes), device=dev), torch.tensor([r * c for r, c, _ in shapes], device=dev))
        if own:
            s["src"] = nshb.tensors(_views(s["flat"], shapes))
            s["ws"] = nshb.tensor_workspace(s["src"])
            s["dst"] = nshb.tensors(_views(s["out"], shapes)) if op == "clip" else None
    elif op == "quantize":
        r, c = case["rows"], case["cols"]
        x = [torch.randn(r, c, generator=gen, device=dev) * math.exp(random.Random(seed + i).uniform(-4, 2)) for i in range(case["count"])]
        s["x"] = [v.to(DTYPE[case["dtype"]]) for v in x]
        if own:
            qr, qc = (c, r) if case["transpose"] else (r, c)
            s["y"] = [torch.empty(qr, qc, dtype=DTYPE[case["dtype"]], device=dev) for _ in x]
            s["src"], s["dst"] = nshb.tensors(s["x"]), nshb.tensors(s["y"])
            s["q"] = nshb.fp4_matrices([nshb.fp4_empty(qr, qc, _format(nshb, case), device=dev) for _ in x])
            s["ws"] = nshb.tensor_workspace(s["src"])
    elif op == "product":
        s["a"] = [_operand(gen, case["m"], case["k"], case["format"], False)]
        s["b"] = [_operand(gen, case["n"], case["k"], case["format"], False)]
        s["d"] = [torch.empty(case["m"], case["n"], dtype=DTYPE[case["out"]], device=dev)]
    else:
        s["a"] = [_operand(gen, case["d"], case["tokens"], case["format"], True) for _ in range(case["count"])]
        s["b"] = None
        s["d"] = [torch.empty(case["d"], case["d"], device=dev) for _ in range(case["count"])]
    if own and op in ("product", "gram"):
        held = lambda side: nshb.fp4_matrices([nshb.Fp4(v["rows"], v["cols"], _format(nshb, case), v["codes"], v["scales"], v["whole"] if case["format"] == "nv" else None) for v in side])  # noqa: E731
        s["A"], s["B"] = held(s["a"]), held(s["b"]) if s["b"] is not None else None
        s["D"] = nshb.tensors(s["d"])
        s["ws"] = nshb.tensor_workspace(s["D"])
    return s


def _format(nshb, case):
    return nshb.NSHB_MXFP4 if case["format"] == "mx" else nshb.NSHB_NVFP4


# --------------------------------------------------------------------------- plain forms


def _plain_norm(s):
    x = s["flat"].float()
    x = x[s["at"]] if "at" in s else x
    sq = x * x
    norm = sq.sum(dtype=torch.float64).sqrt().float()
    return sq, norm, torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)


def _plain_quantize(x, fmt):
    """(magnitude code, sign, scale per block, scale of the whole) of a matrix, blocks along its rows.
    The scale per block is its power of two's exponent ("mx") or its value ("nv")."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, -cols % BLOCK[fmt])).view(rows, -1, BLOCK[fmt])
    top = b.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        whole = torch.ones((), device=x.device)
        scale = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 125)
        b = torch.ldexp(b, -scale)
    else:
        # in 64 bits: a quotient next to the border of two codes must not land on it
        b, top = b.double(), top.double()
        most = torch.frexp(top.amax())
        whole = torch.ldexp(torch.ones((), device=x.device), (most.exponent - 12 + (most.mantissa > 0.65625).int()).clamp(-126, 126))
        whole = torch.where(most.mantissa > 0, whole, 1.0)
        scale = (top / whole / 6).clamp(max=448.0)
        step = torch.ldexp(torch.ones_like(scale), torch.frexp(scale).exponent.clamp(min=-5) - 4)
        scale = torch.round(scale / step) * step
        b = torch.where(scale > 0, b / (scale * whole), torch.copysign(torch.zeros_like(b), b))
        scale = scale.float()
    a = b.abs()
    index = sum(p(a, t).to(torch.uint8) for p, t in ((torch.gt, 0.25), (torch.ge, 0.75), (torch.gt, 1.25), (torch.ge, 1.75), (torch.gt, 2.5), (torch.ge, 3.5), (torch.gt, 5.0)))
    return index.reshape(rows, -1)[:, :cols], torch.signbit(b).to(torch.uint8).reshape(rows, -1)[:, :cols], scale.reshape(rows, -1), whole


def _plain_values(x, fmt):
    """The values that a matrix's 4-bit form stands for."""
    index, sign, scale, whole = _plain_quantize(x.float(), fmt)
    table = torch.tensor(VALUES, device=x.device)
    value = table[index.int()] * (1.0 - 2.0 * sign)
    scale = torch.ldexp(torch.ones(scale.shape, device=x.device), scale) if fmt == "mx" else scale
    return (value * scale.repeat_interleave(BLOCK[fmt], dim=1)[:, :value.shape[1]] * whole).to(x.dtype)


def _plain_operand(v, fmt):
    """A matrix's values without its whole's scale, from its packed codes and tiled scales."""
    rows, cols = v["rows"], v["cols"]
    table = torch.tensor(VALUES + tuple(-x for x in VALUES), device=v["codes"].device)
    values = table[torch.stack((v["codes"] & 15, v["codes"] >> 4), dim=2).int()].reshape(rows, -1)
    wide = values.shape[1] // BLOCK[fmt]
    raw = v["scales"].view(-1, wide // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, wide)[:rows]
    scale = torch.ldexp(torch.ones(raw.shape, device=raw.device), raw.int() - 127) if fmt == "mx" else raw.contiguous().view(torch.float8_e4m3fn).float()
    return (values.view(rows, wide, -1) * scale[:, :, None]).view(rows, -1)[:, :cols]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import newton_schulz_hyperball_b200 as nshb
        if op == "norm":
            nshb.grad_norm(s["src"], s["total"], s["ws"], max_norm=s["max_norm"], each=s.get("each"))
            return (s["total"], s["each"]) if "each" in s else (s["total"],)
        if op == "clip":
            nshb.clip_grads(s["src"], s["max_norm"], s["total"], s["ws"], dst=s["dst"])
            return s["total"], s["out"]
        if op == "quantize":
            nshb.fp4_quantize(s["src"], s["q"], s["ws"], transpose=case["transpose"])
            nshb.fp4_dequantize(s["q"], s["dst"])
            return s["y"]
        nshb.fp4_matmul(s["A"], s["B"], s["D"], s["ws"])
        return s["d"]
    if op == "norm":
        sq, norm, factor = _plain_norm(s)
        total = torch.stack((norm, factor))
        if not case["each"]:
            return (total,)
        each = torch.zeros(s["each"].numel(), dtype=torch.float64, device=sq.device).index_add_(0, s["owner"], sq.double())
        return total, each.sqrt().float()
    if op == "clip":
        _, norm, factor = _plain_norm(s)
        if "at" in s:
            s["out"][s["at"]] = (s["flat"][s["at"]].float() * factor).to(s["out"].dtype)
        else:
            s["out"].copy_(s["flat"].float() * factor)
        return torch.stack((norm, factor)), s["out"]
    if op == "quantize":
        return [_plain_values(x.t() if case["transpose"] else x, case["format"]) for x in s["x"]]
    left = [_plain_operand(v, case["format"]) for v in s["a"]]
    right = left if s["b"] is None else [_plain_operand(v, case["format"]) for v in s["b"]]
    whole = [v["whole"] * w["whole"] for v, w in zip(s["a"], s["b"] or s["a"])]
    return [((x @ y.t()) * g).to(d.dtype) for x, y, g, d in zip(left, right, whole, s["d"])]


# ----------------------------------------------------------------------------- the work


def _bytes_of(rows, cols, fmt):
    return rows * cols / 2 + rows * -(-cols // BLOCK[fmt])


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        n = sum(r * c for r, c, _ in _shapes(case))
        read = n * DTYPE[case["dtype"]].itemsize
        return {"bytes": read + 8, "flops": 2 * n} if op == "norm" else {"bytes": read + n * DTYPE[case["out"]].itemsize + 8, "flops": 3 * n}
    fmt = case["format"]
    if op == "quantize":
        # the round trip: read, 4-bit form written and read, values written
        n, r, c = case["rows"] * case["cols"], case["rows"], case["cols"]
        r, c = (c, r) if case["transpose"] else (r, c)
        return {"bytes": case["count"] * (2 * n * DTYPE[case["dtype"]].itemsize + 2 * _bytes_of(r, c, fmt)), "flops": case["count"] * 4 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _bytes_of(m, k, fmt) + _bytes_of(n, k, fmt) + m * n * DTYPE[case["out"]].itemsize, "flops": 2 * m * n * k}
    d, t = case["d"], case["tokens"]
    return {"bytes": case["count"] * (_bytes_of(d, t, fmt) + 4 * d * d), "flops": case["count"] * d * (d + 1) * t}


# ------------------------------------------------------------------------- in 64 bits


def _exact_round(a):
    """The nearest 4-bit magnitude: steps of 1/2 below 2, of 1 below 4, of 2 above; halves to the even code."""
    return torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6)


def _exact_power(v):
    """The largest power of two that is not over v > 0."""
    return torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent - 1)


def _exact_quantized(x, fmt):
    n, width = x.shape[1], BLOCK[fmt]
    if n % width:
        x = torch.cat((x, x.new_zeros(x.shape[0], width - n % width)), dim=1)
    b = x.reshape(x.shape[0], -1, width)
    top = b.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        unit = _exact_power(top.clamp(min=2.0 ** -125)) / 4
    else:
        most = float(top.max())
        whole = 2.0 ** max(-126, math.ceil(math.log2(most) - math.log2(2688))) if most > 0 else 1.0
        while most > 2688 * whole:
            whole *= 2
        while most <= 1344 * whole and whole > 2.0 ** -126:
            whole /= 2
        grid = torch.tensor([(1 + i % 8 / 8) * 2.0 ** (i // 8 - 7) if i > 7 else i / 8 * 2.0 ** -6 for i in range(127)], dtype=torch.float64, device=x.device)
        v = (top / (6 * whole)).clamp(max=448).contiguous()
        low = torch.searchsorted(grid, v, right=True) - 1
        high = (low + 1).clamp(max=126)
        up = (v - grid[low] > grid[high] - v) | ((v - grid[low] == grid[high] - v) & (low % 2 == 1))
        unit = torch.where(up, grid[high], grid[low]) * whole
    q = torch.sign(b) * _exact_round((b / torch.where(unit > 0, unit, torch.ones_like(unit))).abs())
    return (q * unit).reshape(x.shape[0], -1)[:, :n]


def _exact_operand(v, fmt):
    table = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    out = torch.zeros(v["rows"], v["codes"].shape[1] * 2, dtype=torch.float64, device="cuda")
    for half in (0, 1):
        code = (v["codes"].long() >> (4 * half)) & 15
        out[:, half::2] = table[code % 8] * torch.where(code > 7, -1.0, 1.0)
    width = BLOCK[fmt]
    r = torch.arange(v["rows"], device="cuda")[:, None]
    k = torch.arange(out.shape[1] // width, device="cuda")[None, :]
    at = ((r // 128) * (out.shape[1] // width // 4) + k // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4
    raw = v["scales"][at].double()
    if fmt == "mx":
        scale = 2.0 ** (raw - 127)
    else:
        power, part = torch.floor(raw / 8), raw % 8
        scale = torch.where(power > 0, (1 + part / 8) * 2.0 ** (power - 7), part / 8 * 2.0 ** -6)
    return (out * scale.repeat_interleave(width, dim=1))[:, :v["cols"]] * v["whole"].double()


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("norm", "clip"):
        views, total, each = _views(s["flat"], _shapes(case)), 0.0, []
        for v in views:
            each.append(float(v.double().pow(2).sum()))
        norm = math.sqrt(math.fsum(each))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        total = torch.tensor((norm, factor), dtype=torch.float64)
        if op == "norm":
            return (total, torch.tensor(each, dtype=torch.float64).sqrt()) if case["each"] else (total,)
        out = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        for v, w in zip(views, _views(out, _shapes(case))):
            w.copy_(v.double() * factor)
        return total, out
    if op == "quantize":
        return [_exact_quantized(x.double().t() if case["transpose"] else x.double(), case["format"]) for x in s["x"]]
    left = [_exact_operand(v, case["format"]) for v in s["a"]]
    right = left if s["b"] is None else [_exact_operand(v, case["format"]) for v in s["b"]]
    return [x @ y.t() for x, y in zip(left, right)]
