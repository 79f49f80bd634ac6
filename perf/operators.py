"""The operators around a microscaled (MX) linear layer, case by case.

Formats (OCP Microscaling Formats, MX v1.0): blocks of 32 neighbouring columns share a
power of two 2^(s - 127) held in one byte s (255: the block is NaN); the elements are
e2m1 (4 bits) or e4m3 (8 bits).  Three kinds of buffers hold such a rows x cols matrix:

  codes   rows of ceil(cols / 128) * 128 elements (two e2m1 to a byte, the even column in
          the low half), zero behind the last column;
  scales  one byte per block in tiles of 128 rows x 4 blocks: byte 16 (r % 32) + 4 (r % 128 / 32)
          + k % 4 of tile (r / 128, k / 4), tiles of a row of tiles one after another.

Operators (`op` of a case):

  quantize   a dense matrix (or its transpose) -> codes and scales -> the values they stand for
  forward    y = X W^T of two such matrices, fp32 sums
  norm       h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, y dense or in codes and scales
  norm_bwd   the gradients of the norm for h (with the residual stream's own added) and weight
  layer      norm with its output in codes and scales, and the product that reads it
"""
import torch

own = False

EPS = 1e-5
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
BITS = {"mx4": 4, "mx8": 8}
#: largest exponent, mantissa bits, smallest normal exponent and largest value of the elements
ELEMENT = {"mx4": (2, 1, 0, 6.0), "mx8": (8, 3, -6, 448.0)}


def listed():
    return [
        # a decoder layer's attention weight, brought into 4 bits once when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "rows": 4096, "cols": 4096, "type": "bf16", "fmt": "mx4", "transpose": False},
        # the transpose of an odd gradient block, as the second product of a training step reads it
        {"name": "quantize_transposed", "op": "quantize", "rows": 777, "cols": 1030, "type": "fp32", "fmt": "mx8", "transpose": True},
        # one token's activations in front of a projection: the smallest call, all latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "type": "fp16", "fmt": "mx8", "residual": True},
        # a prompt's activations in front of a projection
        {"name": "norm_prompt", "op": "norm", "rows": 2048, "cols": 4096, "type": "bf16", "fmt": "mx8", "residual": True},
        # dense output at an odd width, for a layer that takes fp16
        {"name": "norm_dense_odd", "op": "norm", "rows": 300, "cols": 5001, "type": "fp16", "fmt": "", "residual": False},
        # gradients of a prompt's norm, the residual stream's gradient arriving too
        {"name": "norm_bwd_prompt", "op": "norm_bwd", "rows": 2048, "cols": 4096, "type": "bf16", "dh": True},
        # few rows of an odd width
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 33, "cols": 1111, "type": "fp32", "dh": False},
        # one token through an attention projection: the weight's bytes and the launch
        {"name": "forward_token", "op": "forward", "batch": 1, "n": 4096, "m_in": 4096, "x": "mx8", "w": "mx4", "type": "fp16"},
        # sixteen tokens through the norm and the wide projection of a decoder layer
        {"name": "layer_tokens", "op": "layer", "batch": 16, "n": 14336, "m_in": 4096, "x": "mx8", "w": "mx4", "type": "bf16"},
        # ragged sizes in every direction, both operands in 8 bits, fp32 results
        {"name": "forward_ragged", "op": "forward", "batch": 77, "n": 1001, "m_in": 1111, "x": "mx8", "w": "mx8", "type": "fp32"},
        # a prompt through the projection back from the wide layer, activations in 8 bits
        {"name": "forward_prompt", "op": "forward", "batch": 2048, "n": 4096, "m_in": 14336, "x": "mx8", "w": "mx4", "type": "bf16"},
        # a prompt through the wide projection, everything in 4 bits: the largest product
        {"name": "forward_wide", "op": "forward", "batch": 2048, "n": 14336, "m_in": 4096, "x": "mx4", "w": "mx4", "type": "fp16"},
    ]


def _log(rng, low, high):
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def _even(rng, size, to):
    """`size` as it is, or rounded up to a multiple of `to`: real widths are even, odd ones have to hold."""
    return -(-size // to) * to if rng.random() < 0.6 else size


def draw(rng):
    op = rng.choice(["quantize", "norm", "norm_bwd", "forward", "forward", "layer"])
    kind = rng.choice(["fp16", "bf16", "fp32"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 8000), _even(rng, _log(rng, 8, 8000), 32)
        return {"op": op, "rows": rows, "cols": cols, "type": kind, "fmt": rng.choice(["mx4", "mx8"]), "transpose": rng.random() < 0.4}
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _even(rng, _log(rng, 32, 16000), 64), "type": kind,
                "fmt": rng.choice(["", "mx4", "mx8", "mx8"]), "residual": rng.random() < 0.7}
    if op == "norm_bwd":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _even(rng, _log(rng, 32, 16000), 64), "type": kind, "dh": rng.random() < 0.7}
    batch, n, m_in = _log(rng, 1, 2048), _even(rng, _log(rng, 16, 14336), 64), _even(rng, _log(rng, 32, 14336), 64)
    batch = max(1, min(batch, 14336 * 4096 * 2048 // (n * m_in)))
    x, w = rng.choice(["mx4", "mx8"]), rng.choice(["mx4", "mx4", "mx8"])
    if op == "layer":  # its product reads rounded values: results in 16 bits, as the layer before and after hold them
        kind = rng.choice(["fp16", "bf16"])
    return {"op": op, "batch": batch, "n": n, "m_in": m_in, "x": x, "w": w, "type": kind}


# ---------------------------------------------------------------- the formats


def _pitch(cols):
    return -(-cols // 128) * 128


def _pow2(e):
    """2^e in fp32 for whole e from -127 to 127, from the bits."""
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantize(v, fmt):
    """The values that `v` (fp32, rows x cols) becomes in the format, over its block's scale, and the exponents of its blocks (255: NaN)."""
    top, mantissa, least, most = ELEMENT[fmt]
    rows, cols = v.shape
    pad = torch.zeros(rows, _pitch(cols), dtype=v.dtype, device=v.device)
    pad[:, :cols] = v
    b = pad.view(rows, -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - top).clamp(-127, 127)  # floor(log2(amax)) - top
    e = torch.where(amax == 0, -127, e)
    u = b * _pow2(-e)
    step = (torch.frexp(u)[1] - 1).clamp(least, top) - mantissa
    q = (torch.round(u * _pow2(-step)) * _pow2(step)).clamp(-most, most)
    bad = ~torch.isfinite(amax)
    e = torch.where(bad, 128, e)
    q = torch.where(bad, 0.0, q)
    return q.view(rows, -1), (e + 127).view(rows, -1)


def _tiles(s):
    """rows x blocks exponents -> the bytes of the scales buffer."""
    rows, blocks = s.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=s.device)
    full[:rows, :blocks] = s.to(torch.uint8)
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(scales, rows, cols):
    """The bytes of the scales buffer -> rows x blocks exponents, as whole numbers."""
    blocks = _pitch(cols) // 32
    t = scales.view(-1, blocks // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, blocks)
    return t[:rows].to(torch.int32)


def _encode(q, fmt):
    """Values on the format's grid -> the bytes of the codes buffer."""
    if fmt == "mx8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)
    a = q.abs()
    c = (2 * a).to(torch.uint8)  # 0, .5, 1, 1.5 -> 0..3
    c = torch.where(a >= 2, (a + 2).to(torch.uint8), c)  # 2, 3 -> 4, 5
    c = torch.where(a >= 4, (a / 2 + 4).to(torch.uint8), c)  # 4, 6 -> 6, 7
    c = c | (torch.signbit(q).to(torch.uint8) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1)


def _decode(codes, scales, rows, cols, fmt):
    """Codes and scales -> the values they stand for, fp32 rows x cols."""
    if fmt == "mx8":
        q = codes.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        c = torch.stack((codes & 15, codes >> 4), 1).reshape(-1).to(torch.int32)
        e, m = (c >> 1) & 3, (c & 1).to(torch.float32)
        q = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _pow2(e - 1))
        q = torch.where(c >= 8, -q, q)
    s = _untile(scales, rows, cols)
    f = torch.where(s == 255, float("nan"), _pow2(s - 127))
    return (q.view(rows, -1, 32) * f[:, :, None]).view(rows, -1)[:, :cols]


# ---------------------------------------------------------------- inputs


def _random(gen, rows, cols):
    return torch.randn(rows, cols, generator=gen, device="cuda")


def _activations(gen, rows, cols):
    """Hidden states: normal, a few columns much larger than the others."""
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.004
    return _random(gen, rows, cols) * torch.where(loud, 20.0, 1.0)


def _held(v, fmt):
    """A matrix as a program keeps it: codes and scales."""
    q, s = _quantize(v, fmt)
    return _encode(q, fmt), _tiles(s)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, op = TYPES[case["type"]], case["op"]
    s = {"case": case}
    if op == "quantize":
        s["src"] = (_random(gen, case["rows"], case["cols"]) * 0.02).to(kind)
        return s
    if op in ("norm", "norm_bwd", "layer"):
        rows, cols = (case["batch"], case["m_in"]) if op == "layer" else (case["rows"], case["cols"])
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(kind)
        s["x"] = _activations(gen, rows, cols).to(kind)
        if op == "norm_bwd":
            s["dy"] = (_random(gen, rows, cols) * 0.01).to(kind)
            s["dh"] = (_random(gen, rows, cols) * 0.01).to(kind) if case["dh"] else None
        else:
            s["residual"] = _activations(gen, rows, cols).to(kind) if op == "layer" or case["residual"] else None
    if op in ("forward", "layer"):
        s["w_codes"], s["w_scales"] = _held(_random(gen, case["n"], case["m_in"]) * 0.02, case["w"])
        if op == "forward":
            s["x_codes"], s["x_scales"] = _held(_activations(gen, case["batch"], case["m_in"]), case["x"])
    if own:
        import binary_factorized_weight_b200 as dbf

        # scratch that a program keeps from call to call
        if op in ("forward", "layer"):
            s["workspace"] = dbf.dbf_mx_new_workspace(case["n"], case["m_in"], case["batch"])
        elif op == "norm_bwd":
            s["workspace"] = dbf.dbf_rmsnorm_backward_new_workspace(case["rows"], case["cols"])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import binary_factorized_weight_b200 as dbf

    c, op = s["case"], s["case"]["op"]
    fmt = {"mx4": dbf.DBF_MX_E2M1, "mx8": dbf.DBF_MX_E4M3, "": None}
    if op == "quantize":
        f, rows, cols = fmt[c["fmt"]], c["rows"], c["cols"]
        codes, scales = dbf.dbf_mx_quantize(s["src"], f, transpose=c["transpose"])
        if c["transpose"]:
            rows, cols = cols, rows
        return dbf.dbf_mx_dequantize(codes, scales, rows, cols, f, dtype=torch.bfloat16)
    if op == "norm" and not c["fmt"]:
        return dbf.dbf_rmsnorm_forward(s["x"], s["weight"], EPS, residual=s["residual"])
    if op == "norm":
        codes, scales, h = dbf.dbf_rmsnorm_mx_forward(s["x"], s["weight"], EPS, fmt[c["fmt"]], residual=s["residual"])
        return dbf.dbf_mx_dequantize(codes, scales, c["rows"], c["cols"], fmt[c["fmt"]], dtype=torch.bfloat16), h
    if op == "norm_bwd":
        return dbf.dbf_rmsnorm_backward(s["dy"], s["x"], s["weight"], EPS, dh=s["dh"], workspace=s["workspace"])
    kind, n, m_in, batch = TYPES[c["type"]], c["n"], c["m_in"], c["batch"]
    h, x_codes, x_scales = None, s.get("x_codes"), s.get("x_scales")
    if op == "layer":
        x_codes, x_scales, h = dbf.dbf_rmsnorm_mx_forward(s["x"], s["weight"], EPS, fmt[c["x"]], residual=s["residual"])
    y = dbf.dbf_mx_forward(x_codes, x_scales, s["w_codes"], s["w_scales"], n, m_in, batch, x_fmt=fmt[c["x"]], w_fmt=fmt[c["w"]],
                           y_dtype=kind, workspace=s["workspace"], flags=dbf.DBF_FWD_WEIGHTS_STATIC)
    return y if op == "forward" else (y, h)


def _norm(s, h):
    v = h.float()
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["weight"].float()


def _values(v, fmt):
    q, e = _quantize(v, fmt)
    f = torch.where(e == 255, float("nan"), _pow2(e - 127))
    return (q.view(q.shape[0], -1, 32) * f[:, :, None]).view(q.shape)[:, : v.shape[1]]


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    kind = TYPES[c["type"]]
    if op == "quantize":
        v = s["src"].float()
        return _values(v.t().contiguous() if c["transpose"] else v, c["fmt"]).to(torch.bfloat16)
    if op in ("norm", "layer"):
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(kind)
        y = _norm(s, h)
        if op == "norm":
            return (_values(y, c["fmt"]).to(torch.bfloat16) if c["fmt"] else y.to(kind)), h
        return (_values(y, c["x"]) @ _decode(s["w_codes"], s["w_scales"], c["n"], c["m_in"], c["w"]).t()).to(kind), h
    if op == "norm_bwd":
        h, g = s["x"].float(), s["dy"].float() * s["weight"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dx.to(kind), (s["dy"].float() * h * r).sum(0)
    x = _decode(s["x_codes"], s["x_scales"], c["batch"], c["m_in"], c["x"])
    return (x @ _decode(s["w_codes"], s["w_scales"], c["n"], c["m_in"], c["w"]).t()).to(kind)


# ---------------------------------------------------------------- what a pass cannot do without


def _bytes_held(rows, cols, fmt):
    return rows * _pitch(cols) * BITS[fmt] // 8 + rows * _pitch(cols) // 32


def work(case):
    op, size = case["op"], SIZE[case["type"]]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return {"bytes": n * size + _bytes_held(r, c, case["fmt"]) + 2 * n, "flops": 4 * n}
    if op == "norm":
        n = case["rows"] * case["cols"]
        read = n * size * (2 if case["residual"] else 1) + case["cols"] * size
        wrote = (n * size if case["residual"] else 0) + (_bytes_held(case["rows"], case["cols"], case["fmt"]) + 2 * n if case["fmt"] else n * size)
        return {"bytes": read + wrote, "flops": 5 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (4 if case["dh"] else 3) + case["cols"] * (size + 4), "flops": 12 * n}
    b, n, m = case["batch"], case["n"], case["m_in"]
    bytes_ = _bytes_held(n, m, case["w"]) + b * n * size
    bytes_ += 3 * b * m * size + m * size if op == "layer" else _bytes_held(b, m, case["x"])
    return {"bytes": bytes_, "flops": 2 * b * n * m}


# ---------------------------------------------------------------- the definition in 64 bits


def _table(fmt):
    """The value of each code, from the bits: sign, exponent, mantissa."""
    total, mantissa, bias = (4, 1, 1) if fmt == "mx4" else (8, 3, 7)
    out = []
    for code in range(1 << total):
        e, m = (code & ((1 << (total - 1)) - 1)) >> mantissa, code & ((1 << mantissa) - 1)
        v = m * 2.0 ** (1 - bias - mantissa) if e == 0 else (1 + m / (1 << mantissa)) * 2.0 ** (e - bias)
        out.append(-v if code >> (total - 1) else v)
    if fmt == "mx8":
        out[0x7F] = out[0xFF] = float("nan")
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_held(codes, scales, rows, cols, fmt):
    c = codes.long()
    if fmt == "mx4":
        c = torch.stack((c % 16, c // 16), -1)
    q = _table(fmt)[c.reshape(rows, -1)[:, :cols]]
    r, k = torch.arange(rows, device="cuda")[:, None], (torch.arange(cols, device="cuda") // 32)[None, :]
    at = ((r // 128) * (_pitch(cols) // 128) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    s = scales[at].double()
    return torch.where(s == 255, float("nan"), q * 2.0 ** (s - 127))


def _exact_rounded(v, fmt):
    """The nearest values of the format (ties to the even code), by search in the table of its values."""
    rows, cols = v.shape
    grid = _table(fmt)[: 0x7F if fmt == "mx8" else 8]  # the codes 0, 1, .. without sign, in order
    pad = torch.nn.functional.pad(v, (0, -cols % 32)).view(rows, -1, 32)
    most = pad.abs().amax(-1)
    scale = 2.0 ** (torch.floor(torch.log2(most.clamp(min=2.0 ** -140))) - ELEMENT[fmt][0]).clamp(-127, 127)
    scale = torch.where(torch.isfinite(most), scale, float("nan"))[:, :, None]
    u = pad.abs() / scale
    up = torch.searchsorted(grid, u.contiguous()).clamp(1, len(grid) - 1)
    low, high = grid[up - 1], grid[up]
    code = torch.where((u - low < high - u) | ((u - low == high - u) & (up % 2 == 1)), up - 1, up)
    return (torch.where(pad < 0, -1.0, 1.0) * grid[code] * scale).view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v = s["src"].double()
        return _exact_rounded(v.t() if case["transpose"] else v, case["fmt"])
    if op in ("norm", "layer"):
        total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        h = total.to(s["x"].dtype).double()  # h is rounded to its type before the norm reads it
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double()
        if op == "norm":
            return (_exact_rounded(y, case["fmt"]) if case["fmt"] else y), total
        w = _exact_held(s["w_codes"], s["w_scales"], case["n"], case["m_in"], case["w"])
        return torch.matmul(_exact_rounded(y, case["x"]), w.t()), total
    if op == "norm_bwd":
        h = s["x"].double().requires_grad_()
        w = s["weight"].double().requires_grad_()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + EPS) * w
        dx, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return dx if s["dh"] is None else dx + s["dh"].double(), dw
    x = _exact_held(s["x_codes"], s["x_scales"], case["batch"], case["m_in"], case["x"])
    return torch.matmul(x, _exact_held(s["w_codes"], s["w_scales"], case["n"], case["m_in"], case["w"]).t())
