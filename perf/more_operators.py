"""What is measured of the operators of the feed-forward half of a block.

Three operators (`op`): "gated", both projections of a gated feed-forward
block from NVFP4 operands with the activation and the product, and its
backward pass from the output gradient's and the down projection's operands;
"norm", the norms after and before a block with its gate and residual scale,
forward and backward; "ckpt", activations kept in 8 bits and brought back.
`listed()` holds the named cases, `draw()` makes more of the same ranges;
`run()` computes either the plain form (elementary torch operations in 32
bits) or, where `own` is true, the framework's kernels on the same inputs;
`exact()` is the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
GELU_SLOPE, GELU_CUBE = 2 * math.sqrt(2 / math.pi), 0.044715


def _gated(name, tokens, hidden, ffn, act, train, keep):
    return {"name": name, "op": "gated", "tokens": tokens, "hidden": hidden, "ffn": ffn, "act": act, "train": train,
            "keep": keep}


def _norm(name, tokens, width, train, post, gate, scale=1.0, fp32=False, keep="bf16"):
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "train": train, "post": post, "gate": gate,
            "scale": scale, "fp32": fp32, "keep": keep}


def _ckpt(name, rows, cols, spare):
    return {"name": name, "op": "ckpt", "rows": rows, "cols": cols, "spare": spare}


def listed():
    return [
        # one token through the 3B model's feed-forward projections: latency, bound by the weights
        _gated("gated_1", 1, 3072, 9216, "silu", False, "none"),
        # forward of 4 sequences of 2048 tokens without a backward pass
        _gated("gated_8192", 8192, 3072, 9216, "silu", False, "none"),
        # a training step's batch, gate and up kept in BF16 for the backward pass
        _gated("gated_train_16384", 16384, 3072, 9216, "silu", True, "bf16"),
        # the same batch with gate and up kept in 8 bits
        _gated("gated_train_16384_8bit", 16384, 3072, 9216, "silu", True, "e4m3"),
        # a small model, sizes that fill no tile
        _gated("gated_train_odd", 1003, 1040, 2736, "gelu", True, "e4m3"),
        # one token through the norms of a block
        _norm("norm_1", 1, 3072, False, True, "channel"),
        # pre-norm residual stream, forward of 4 sequences
        _norm("norm_8192", 8192, 3072, False, False, "none"),
        # a training step's batch: norms before and after, a gate per channel
        _norm("norm_train_16384", 16384, 3072, True, True, "channel", 0.75),
        # FP32 residual stream, a gate per token and channel, odd sizes, the branch kept in 8 bits
        _norm("norm_train_odd", 4099, 2056, True, True, "token", 0.9, True, "e4m3"),
        # a short batch's activations kept in 8 bits
        _ckpt("ckpt_512", 512, 1024, 0),
        # columns of a wider matrix, an odd number of rows, a last block that is not full
        _ckpt("ckpt_odd", 5003, 1000, 488),
        # a training step's feed-forward activations
        _ckpt("ckpt_16384", 16384, 9216, 0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.45:
        train = rng.random() < 0.6
        c = _gated("", _log_int(rng, 1, 16384), 16 * _log_int(rng, 16, 192), 16 * _log_int(rng, 16, 576),
                   rng.choice(["silu", "silu", "gelu"]), train, rng.choice(["bf16", "e4m3"]) if train else "none")
    elif kind < 0.8:
        width = 8 * _log_int(rng, 8, 1024)
        c = _norm("", _log_int(rng, 1, min(16384, 16384 * 3072 // width)), width, rng.random() < 0.6,
                  rng.random() < 0.6, rng.choice(["none", "channel", "token"]), rng.choice([1.0, 0.75, 0.5]),
                  rng.random() < 0.4, rng.choice(["bf16", "e4m3"]))
    else:
        c = _ckpt("", _log_int(rng, 1, 16384), 8 * _log_int(rng, 8, 1152), 8 * rng.choice([0, 0, 1, 37]))
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _gradient(gen, *shape):
    """Output gradients as in training: Student-t with 3 degrees of freedom, times 1e-3."""
    chi = _normal(gen, *shape).square_()
    for _ in range(2):
        chi += _normal(gen, *shape).square_()
    return _normal(gen, *shape) / (chi / 3).sqrt_() * 1e-3


def _outliers(gen, x):
    """Activations: one channel in a thousand 50 times as large."""
    x[:, torch.randint(0, x.shape[1], (max(1, x.shape[1] // 1000),), generator=gen, device="cuda")] *= 50
    return x


def _nvfp4(x, tile=False):
    """x [rows][cols] as an NVFP4 operand in the layout that the framework documents: codes two per byte, E4M3
    scales of 1x16 blocks (or of 16x16 tiles) in 128-row x 4-scale tiles, the FP32 scale of the tensor."""
    rows, cols = x.shape
    blocks = x.view(rows, cols // 16, 16)
    amax_b = blocks.abs().amax(-1)
    amax = amax_b.max()
    if tile:
        pad = (-rows) % 16
        t = torch.cat([amax_b, amax_b.new_zeros(pad, amax_b.shape[1])]).view(-1, 16, amax_b.shape[1]).amax(1)
        amax_b = t.repeat_interleave(16, 0)[:rows]
    enc = 2688 / amax
    s = (amax_b / 6 * enc).to(torch.float8_e4m3fn)
    sf = s.float()
    v = blocks * torch.where(sf == 0, 0.0, enc / sf)[..., None]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(v.abs(), ties).to(torch.uint8) + 8 * torch.signbit(v).to(torch.uint8)
    code = code.view(rows, cols // 2, 2)
    codes = torch.zeros(rows, (cols // 2 + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    codes[:, :cols // 2] = code[..., 0] | (code[..., 1] << 4)
    r, g = (rows + 127) // 128, (cols + 63) // 64
    padded = torch.zeros(r * 128, g * 4, dtype=torch.uint8, device="cuda")
    padded[:rows, :cols // 16] = s.view(torch.uint8)
    scales = padded.view(r, 4, 32, g, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return {"codes": codes, "scales": scales, "amax": amax.view(1), "global_scale": (1 / enc).view(1), "rows": rows,
            "cols": cols}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] == "gated":
        m, k, n = case["tokens"], case["hidden"], case["ffn"]
        s["x"] = _nvfp4(_outliers(gen, _normal(gen, m, k)))
        s["wg"] = _nvfp4(0.02 * _normal(gen, n, k), True)
        s["wu"] = _nvfp4(0.02 * _normal(gen, n, k), True)
        if case["train"]:
            # the output gradient's row-wise operand and the down projection's col-wise one
            s["dy"] = _nvfp4(_gradient(gen, m, k))
            s["wd"] = _nvfp4(0.02 * _normal(gen, n, k), True)
    elif case["op"] == "norm":
        t, h = case["tokens"], case["width"]
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        s["residual"] = _outliers(gen, 4 * _normal(gen, t, h)).to(kind)
        s["branch"] = _outliers(gen, 0.5 * _normal(gen, t, h)).to(torch.bfloat16)
        s["pre"] = 1 + 0.1 * _normal(gen, h)
        s["post"] = 1 + 0.1 * _normal(gen, h) if case["post"] else None
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = 0.5 + 0.1 * _normal(gen, h)
        elif case["gate"] == "token":
            s["gate"] = torch.sigmoid(_normal(gen, t, h)).to(torch.bfloat16)
        if case["train"]:
            # what the forward pass left for the backward pass, and the gradients that reach it
            s["kept"] = _norm_forward_plain(s, case)[0]
            s["codes"], s["scales"] = _encode_plain(s["branch"]) if case["keep"] == "e4m3" else (None, None)
            s["dresidual"] = _gradient(gen, t, h).to(kind)
            s["dnormed"] = _gradient(gen, t, h).to(torch.bfloat16)
    else:
        x = _outliers(gen, _normal(gen, case["rows"], case["cols"] + case["spare"])).to(torch.bfloat16)
        s["x"] = x[:, :case["cols"]]
    return s


# ---- the framework's calls ------------------------------------------------
def _operand(o):
    from fp4_gemm_nvfp4_gb300 import ops
    return ops.NVFP4Operand(o["codes"], o["scales"], o["amax"], o["global_scale"], o["rows"], o["cols"])


def _gated_own(s, c):
    from fp4_gemm_nvfp4_gb300 import ops
    keep = None if c["keep"] == "none" else c["keep"]
    h, gate, up = ops.gemm_gated(_operand(s["x"]), _operand(s["wg"]), _operand(s["wu"]), activation=c["act"], keep=keep)
    if not c["train"]:
        return {"h": h}
    return {"h": h, "dgu": ops.gemm_gated_backward(_operand(s["dy"]), _operand(s["wd"]), gate, up, activation=c["act"])}


def _norm_own(s, c):
    from fp4_gemm_nvfp4_gb300 import ops
    keep = "e4m3" if c["train"] and c["keep"] == "e4m3" else None
    args = {"pre_weight": s["pre"], "post_weight": s["post"], "gate": s["gate"], "residual_scale": c["scale"], "eps": EPS}
    residual, normed, kept = ops.block_norm(s["residual"], s["branch"], keep=keep, **args)
    out = {"residual": residual, "normed": normed}
    if not c["train"]:
        return out
    branch = s["branch"]
    if keep:
        out["codes"], out["scales"] = kept.data[:, :c["width"]].view(torch.float8_e4m3fn), kept.scales[:, :(c["width"] + 31) // 32]
        branch = ops.Checkpoint(s["codes"], s["scales"], c["tokens"], c["width"])
    g = ops.block_norm_backward(s["dresidual"], s["dnormed"], s["kept"], branch, **args)
    out |= {"dresidual": g.dresidual, "dbranch": g.dbranch, "dpre": g.dpre_weight}
    if c["post"]:
        out["dpost"] = g.dpost_weight
    if c["gate"] != "none":
        out["dgate"] = g.dgate
    return out


def _ckpt_own(s, c):
    from fp4_gemm_nvfp4_gb300 import ops
    kept = ops.checkpoint_encode(s["x"])
    return {"x": ops.checkpoint_decode(kept), "scales": kept.scales[:, :(c["cols"] + 31) // 32]}


# ---- the plain forms ------------------------------------------------------
def _dequantize(o):
    rows, cols = o["rows"], o["cols"]
    r, g = (rows + 127) // 128, (cols + 63) // 64
    scales = o["scales"].view(r, g, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, g * 4)[:rows, :cols // 16]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    grid = torch.cat([grid, -grid])
    codes = o["codes"][:, :cols // 2]
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).view(rows, cols // 16, 16)
    return (v * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]).view(rows, cols) * o["global_scale"]


def _exponents(x):
    """Per 1x32 block of x (FP32) the biased exponent of the smallest power of two that takes its largest magnitude
    to at most 448."""
    cols = x.shape[1]
    pad = torch.cat([x, x.new_zeros(x.shape[0], -cols % 32)], 1)
    bits = pad.view(x.shape[0], -1, 32).abs().amax(-1).view(torch.int32)
    return torch.clamp(((bits + 0x1FFFFF) >> 23) - 8, min=10)


def _powers(e, cols):
    return (e << 23).view(torch.float32).repeat_interleave(32, 1)[:, :cols]


def _encode_plain(x):
    """x in 8 bits as the framework keeps it: E4M3 codes and scale bytes, rows of whole 16-byte pieces."""
    rows, cols = x.shape
    x = x.float()
    e = _exponents(x)
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    codes[:, :cols] = (x / _powers(e, cols)).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.zeros(rows, (e.shape[1] + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    scales[:, :e.shape[1]] = e
    return codes, scales


def _decode_plain(codes, scales, cols):
    e = scales[:, :(cols + 31) // 32].int()
    return codes[:, :cols].contiguous().view(torch.float8_e4m3fn).float() * _powers(e, cols)


def _kept_plain(x, keep):
    """What comes back of a value kept for the backward pass."""
    return x.to(torch.bfloat16).float() if keep == "bf16" else _decode_plain(*_encode_plain(x), x.shape[1])


def _sigmoid_of(g, act):
    """The activation is g times this; and the derivative of what the sigmoid is taken of."""
    if act == "silu":
        return 1 / (1 + torch.exp(-g)), 1.0
    return 1 / (1 + torch.exp(-GELU_SLOPE * (g + GELU_CUBE * g * g * g))), GELU_SLOPE * (1 + 3 * GELU_CUBE * g * g)


def _gated_plain(s, c):
    x = _dequantize(s["x"])
    g, u = x @ _dequantize(s["wg"]).t(), x @ _dequantize(s["wu"]).t()
    sg, _ = _sigmoid_of(g, c["act"])
    out = {"h": (g * sg * u).to(torch.bfloat16)}
    if c["train"]:
        dh = _dequantize(s["dy"]) @ _dequantize(s["wd"]).t()
        g, u = _kept_plain(g, c["keep"]), _kept_plain(u, c["keep"])
        sg, slope = _sigmoid_of(g, c["act"])
        out["dgu"] = torch.cat([dh * u * (sg + g * sg * (1 - sg) * slope), dh * g * sg], 1).to(torch.bfloat16)
    return out


def _norm_forward_plain(s, c):
    h = s["branch"].float()
    if c["post"]:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["post"]
    if c["gate"] != "none":
        h = h * s["gate"].float()
    r = (s["residual"].float() * c["scale"] + h).to(s["residual"].dtype)
    x = r.float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["pre"]
    return r, n.to(torch.bfloat16)


def _norm_plain(s, c):
    residual, normed = _norm_forward_plain(s, c)
    out = {"residual": residual, "normed": normed}
    if not c["train"]:
        return out
    y = s["branch"].float()
    if c["keep"] == "e4m3":
        codes, scales = _encode_plain(s["branch"])
        out["codes"], out["scales"] = codes[:, :c["width"]].view(torch.float8_e4m3fn), scales[:, :(c["width"] + 31) // 32]
        y = _decode_plain(s["codes"], s["scales"], c["width"])
    x, dn = s["kept"].float(), s["dnormed"].float()
    rq = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, g = x * rq, dn * s["pre"]
    d = s["dresidual"].float() + rq * (g - xh * (g * xh).mean(-1, keepdim=True))
    out["dpre"] = (dn * xh).sum(0)
    out["dresidual"] = (d * c["scale"]).to(s["residual"].dtype)
    gate = 1.0 if c["gate"] == "none" else s["gate"].float()
    rp = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    a = y * rp
    h = a * s["post"] if c["post"] else y
    if c["gate"] == "channel":
        out["dgate"] = (d * h).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (d * h).to(torch.bfloat16)
    dh = d * gate
    if c["post"]:
        out["dpost"] = (dh * a).sum(0)
        t = dh * s["post"]
        dh = rp * (t - a * (t * a).mean(-1, keepdim=True))
    out["dbranch"] = dh.to(torch.bfloat16)
    return out


def _ckpt_plain(s, c):
    codes, scales = _encode_plain(s["x"])
    return {"x": _decode_plain(codes, scales, c["cols"]).to(torch.bfloat16), "scales": scales[:, :(c["cols"] + 31) // 32]}


def run(state):
    c = state["case"]
    if c["op"] == "gated":
        return (_gated_own if own else _gated_plain)(state, c)
    if c["op"] == "norm":
        return (_norm_own if own else _norm_plain)(state, c)
    return (_ckpt_own if own else _ckpt_plain)(state, c)


# ---- what a pass cannot do without ----------------------------------------
def work(case):
    if case["op"] == "gated":
        m, k, n = case["tokens"], case["hidden"], case["ffn"]
        kept = {"none": 0, "bf16": 4, "e4m3": 2 + 1 / 16}[case["keep"]] * m * n
        forward = {"bytes": 0.5625 * k * (m + 2 * n) + 2 * m * n + kept, "flops": 4 * m * n * k}
        if not case["train"]:
            return forward
        # backward: the gradient's and the down projection's operands, gate and up in, both gradients out
        return {"bytes": forward["bytes"] + 0.5625 * k * (m + n) + kept + 4 * m * n, "flops": forward["flops"] + 2 * m * n * k}
    if case["op"] == "norm":
        t, h = case["tokens"], case["width"]
        r = 4 if case["fp32"] else 2
        vectors = 4 * h * (1 + case["post"] + (case["gate"] == "channel"))
        token = 2 if case["gate"] == "token" else 0
        forward = t * h * (2 * r + 4 + token) + vectors
        if not case["train"]:
            return {"bytes": forward, "flops": 10 * t * h}
        y = 33 / 32 if case["keep"] == "e4m3" else 2
        if case["keep"] == "e4m3":
            forward += t * h * y
        # backward: both gradients, the kept residual and branch in, two gradients out, and the weights' ones
        return {"bytes": forward + t * h * (3 * r + 4 + y + 2 * token) + 2 * vectors, "flops": 40 * t * h}
    n = case["rows"] * case["cols"]
    return {"bytes": n * (4 + 2 * 33 / 32), "flops": 6 * n}


# ---- the definitions in 64 bits -------------------------------------------
def _exact_operand(o):
    """The values of an NVFP4 operand by the format's definition."""
    rows, cols = o["rows"], o["cols"]
    r = torch.arange(rows, device="cuda")[:, None]
    j = torch.arange(cols // 16, device="cuda")[None]
    at = (r // 128 * ((cols + 63) // 64) + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4
    b = o["scales"][at].long()
    e, m = (b >> 3) & 15, (b & 7).double()
    scale = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    value = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    for half in (0, 1):
        q = (o["codes"][:, :cols // 2].long() >> (4 * half)) & 15
        e, m = (q >> 1) & 3, (q & 1).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
        value[:, half::2] = torch.where(q >= 8, -v, v)
    return (value.view(rows, -1, 16) * scale[..., None]).view(rows, cols) * o["global_scale"].double()


def _exact_steps(v, bits, least):
    """v at the nearest value with `bits` bits after the leading one (ties to even) and no step under 2^least."""
    e = torch.frexp(v)[1].double() - 1 - bits
    step = torch.exp2(e.clamp(min=least))
    return torch.round(v / step) * step


def _exact_scale(x):
    """Per column the power of two of its 1x32 block, and its exponent per block."""
    blocks = [c.abs().amax(1) for c in x.split(32, 1)]
    amax = torch.stack(blocks, 1)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -150) / 448)).clamp(min=-117)
    # the logarithm may be off by its last bit
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((amax <= 448 * torch.exp2(e - 1)) & (e > -117), e - 1, e)
    return torch.exp2(e).repeat_interleave(32, 1)[:, :x.shape[1]], e


def _exact_kept(x, keep):
    if keep == "bf16":
        return _exact_steps(x, 7, -133)
    scale, _ = _exact_scale(x)
    return _exact_steps(x / scale, 3, -9) * scale


def _exact_act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    th = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    inner = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * inner


def _gated_exact(s, c):
    x = _exact_operand(s["x"])
    g, u = x @ _exact_operand(s["wg"]).t(), x @ _exact_operand(s["wu"]).t()
    out = {"h": _exact_act(g, c["act"])[0] * u}
    if c["train"]:
        dh = _exact_operand(s["dy"]) @ _exact_operand(s["wd"]).t()
        f, df = _exact_act(_exact_kept(g, c["keep"]), c["act"])
        out["dgu"] = torch.cat([dh * _exact_kept(u, c["keep"]) * df, dh * f], 1)
    return out


def _norm_exact(s, c):
    def over(x):
        return (x.pow(2).sum(-1, keepdim=True) / x.shape[1] + EPS).sqrt()

    h = y = s["branch"].double()
    if c["post"]:
        h = y / over(y) * s["post"].double()
    gate = s["gate"].double() if c["gate"] != "none" else torch.ones_like(h)
    residual = s["residual"].double() * c["scale"] + gate * h
    seen = residual if c["fp32"] else _exact_steps(residual, 7, -133)
    out = {"residual": residual, "normed": seen / over(seen) * s["pre"].double()}
    if not c["train"]:
        return out
    if c["keep"] == "e4m3":
        scale, e = _exact_scale(y)
        out["codes"], out["scales"] = y / scale, (e + 127).to(torch.uint8)
        y = _exact_kept(y, "e4m3")
    x, dn, w = s["kept"].double(), s["dnormed"].double(), s["pre"].double()
    size = over(x)
    along = torch.einsum("th,th->t", dn * w, x)[:, None]
    d = s["dresidual"].double() + dn * w / size - x * along / (x.shape[1] * size.pow(3))
    out["dpre"] = torch.einsum("th,th->h", dn, x / size)
    out["dresidual"] = d * c["scale"]
    size = over(y)
    h = y / size * s["post"].double() if c["post"] else y
    if c["gate"] == "channel":
        out["dgate"] = torch.einsum("th,th->h", d, h)
    elif c["gate"] == "token":
        out["dgate"] = d * h
    dh = d * gate
    if c["post"]:
        out["dpost"] = torch.einsum("th,th->h", dh, y / size)
        dh = dh * s["post"].double()
        along = torch.einsum("th,th->t", dh, y)[:, None]
        dh = dh / size - y * along / (y.shape[1] * size.pow(3))
    out["dbranch"] = dh
    return out


def _ckpt_exact(s, c):
    x = s["x"].double()
    return {"x": _exact_kept(x, "e4m3"), "scales": (_exact_scale(x)[1] + 127).to(torch.uint8)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _gated_exact, "norm": _norm_exact, "ckpt": _ckpt_exact}[case["op"]](s, case)
