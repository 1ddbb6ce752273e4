"""What is measured of the operators between the QKV and the O projection.

Two operators, forward and backward: the per-head RMS norm of queries and
keys with the position rotation (`op` "rope"), and grouped-query attention
with an optional tanh cap, distance bias, document and prefix mask (`op`
"attn").  `listed()` holds the named cases, `draw()` makes more of the same
ranges; `run()` computes either the plain form (elementary torch operations
in 32 bits) or, where `own` is true, the framework's kernels on the same
inputs; `exact()` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0


def _rope(name, tokens, q_heads, kv_heads, dim, rot, interleaved, train):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved, "train": train}


def _attn(name, tokens, q_heads, kv_heads, dim, train, doc, ragged=False, pad=0, causal=True, prefix=False, cap=0.0,
          bias=False):
    return {"name": name, "op": "attn", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "train": train, "doc": doc, "ragged": ragged, "pad": pad, "causal": causal, "prefix": prefix, "cap": cap,
            "bias": bias}


def listed():
    return [
        # one token through the 3B model's heads (24 query, 12 key/value heads of 128): latency
        _rope("rope_1", 1, 24, 12, 128, 128, False, False),
        # the forward pass of a batch of 4 x 2048 tokens, the 3B model's attention configuration
        _rope("rope_8192", 8192, 24, 12, 128, 128, False, False),
        # a whole training step's batch of 16384 tokens, forward and backward
        _rope("rope_train_16384", 16384, 24, 12, 128, 128, False, True),
        # a small model, an odd number of tokens, half of each head rotated, neighbouring pairs
        _rope("rope_train_odd", 4099, 8, 2, 64, 32, True, True),
        # one token: the shortest sequence there is
        _attn("attn_1", 1, 24, 12, 128, False, 1),
        # a short prompt, bidirectional documents packed into one batch, small heads
        _attn("attn_train_short", 500, 16, 16, 64, True, 120, ragged=True, causal=False),
        # forward of 4 sequences of the model's context length
        _attn("attn_4x2048", 8192, 24, 12, 128, False, 2048),
        # training on the same batch
        _attn("attn_train_4x2048", 8192, 24, 12, 128, True, 2048),
        # training on packed documents with a bidirectional prefix each and a padded end of the batch
        _attn("attn_train_docs", 5003, 8, 2, 64, True, 700, ragged=True, pad=37, prefix=True),
        # forward of one long sequence with capped scores
        _attn("attn_cap_8192", 8192, 16, 4, 128, False, 8192, cap=30.0),
        # training with cap and distance bias: an odd length, an odd number of heads, a head size between the tiles'
        _attn("attn_train_bias_odd", 2047, 5, 1, 96, True, 2047, cap=50.0, bias=True),
        # training on one sequence of four times the context length: the most work
        _attn("attn_train_8192", 8192, 24, 12, 128, True, 8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        q, kv = rng.choice([(24, 12), (16, 4), (8, 2), (5, 1), (12, 12), (7, 7)])
        dim = rng.choice([32, 64, 80, 96, 128])
        c = _rope("", _log_int(rng, 1, 16384), q, kv, dim, rng.randrange(0, dim // 16 + 1) * 16, rng.random() < 0.4,
                  rng.random() < 0.6)
    else:
        q, kv = rng.choice([(24, 12), (16, 4), (8, 2), (5, 1), (6, 6), (9, 3)])
        tokens = _log_int(rng, 1, 8192)
        doc = tokens if rng.random() < 0.3 else _log_int(rng, min(tokens, 16), tokens)
        causal = rng.random() < 0.75
        c = _attn("", tokens, q, kv, rng.choice([32, 64, 80, 96, 128]), rng.random() < 0.6, doc,
                  ragged=rng.random() < 0.6, pad=rng.choice([0, 0, rng.randrange(0, tokens // 8 + 1)]), causal=causal,
                  prefix=causal and rng.random() < 0.3, cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]),
                  bias=rng.random() < 0.3)
    del c["name"]
    return c


def _documents(case):
    """[(start, end, prefix)] of the case's documents: a layout of its own, the same for every seed."""
    rng = random.Random("%d/%d/%d" % (case["tokens"], case["doc"], case["pad"]))
    at, end, docs = 0, case["tokens"] - case["pad"], []
    while at < end:
        n = case["doc"]
        if case["ragged"]:
            n = max(1, int(rng.expovariate(1.0) * n))
        n = min(n, end - at)
        docs.append((at, at + n, int(rng.random() * n) if case["prefix"] else 0))
        at += n
    return docs


def _spans(case):
    """Per token the keys it attends to, [first, one past the last): empty for the padding after the documents."""
    lo, hi = [], []
    for start, end, prefix in _documents(case):
        for i in range(start, end):
            lo.append(start)
            hi.append(max(i + 1, start + prefix) if case["causal"] else end)
    rest = case["tokens"] - len(lo)
    return lo + [0] * rest, hi + [0] * rest


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _gradient(gen, *shape):
    """Output gradients as in training: Student-t with 3 degrees of freedom, times 1e-3."""
    chi = _normal(gen, *shape).square_()
    for _ in range(2):
        chi += _normal(gen, *shape).square_()
    return (_normal(gen, *shape) / (chi / 3).sqrt_() * 1e-3).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    t, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    s = {"case": dict(case), "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "rope":
        # the QKV projection's output; a few channels are larger, as activations' are
        x = _normal(gen, t, (hq + 2 * hkv) * d)
        x[:, torch.randint(0, x.shape[1], (max(1, x.shape[1] // 1000),), generator=gen, device="cuda")] *= 50
        s["qkv"] = x.to(torch.bfloat16)
        s["wq"] = 1 + 0.1 * _normal(gen, d)
        s["wk"] = 1 + 0.1 * _normal(gen, d)
        # positions of sequences of 2048 tokens that start anywhere
        start = int(torch.randint(0, 2048, (1,), generator=gen, device="cuda"))
        s["positions"] = ((torch.arange(t, device="cuda") + start) % 2048).to(torch.int32)
        f = BASE ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / max(1, case["rot"]))
        a = torch.arange(2048, device="cuda", dtype=torch.float64)[:, None] * f
        s["cos"], s["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
        if case["train"]:
            s["dq"], s["dk"] = _gradient(gen, t, hq, d), _gradient(gen, t, hkv, d)
        return s

    def unit(h):
        x = _normal(gen, t, h, d)
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True)) * (1.3 + 0.1 * _normal(gen, d))).to(torch.bfloat16)

    s["q"], s["k"] = unit(hq), unit(hkv)
    # the values stay where the QKV projection wrote them: the last columns of its output
    s["v"] = _normal(gen, t, (hq + 2 * hkv) * d).to(torch.bfloat16)[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    lo, hi = _spans(case)
    s["spans"] = torch.tensor([lo, hi], dtype=torch.int32).t().contiguous().cuda()
    s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)) if case["bias"] else None
    if case["train"]:
        s["do"] = _gradient(gen, t, hq, d)
    return s


def _rope_own(s, c):
    from fp4_gemm_nvfp4_gb300 import ops
    q, k = ops.qk_norm_rope(s["qkv"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], q_heads=c["q_heads"],
                            kv_heads=c["kv_heads"], eps=EPS, interleaved=c["interleaved"])
    if not c["train"]:
        return {"q": q, "k": k}
    dqk, dwq, dwk = ops.qk_norm_rope_backward(s["dq"], s["dk"], s["qkv"], s["wq"], s["wk"], s["cos"], s["sin"],
                                              s["positions"], eps=EPS, interleaved=c["interleaved"])
    return {"q": q, "k": k, "dqk": dqk, "dwq": dwq, "dwk": dwk}


def _attn_own(s, c):
    from fp4_gemm_nvfp4_gb300 import ops
    o, lse = ops.attention(s["q"], s["k"], s["v"], s["spans"], scale=s["scale"], softcap=c["cap"], slopes=s["slopes"])
    if not c["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv = ops.attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse, s["spans"], scale=s["scale"],
                                        softcap=c["cap"], slopes=s["slopes"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _rotate(x, cos, sin, interleaved):
    """x [tokens][heads][dim] with the first 2 * cos.shape[-1] dims turned by the angle of each token."""
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _norm_rotate(x, w, cos, sin, interleaved):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _rotate(n, cos, sin, interleaved).to(torch.bfloat16)


def _norm_rotate_gradient(dy, x, w, cos, sin, interleaved):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dn = _rotate(dy.float(), cos, -sin, interleaved)
    xh = x * r
    g = dn * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dn * xh).sum((0, 1))


def _rope_plain(s, c):
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    x = s["qkv"][:, :(hq + hkv) * d].float().unflatten(1, (hq + hkv, d))
    xq, xk = x[:, :hq], x[:, hq:]
    p = s["positions"].long()
    cos, sin = s["cos"][p], s["sin"][p]
    out = {"q": _norm_rotate(xq, s["wq"], cos, sin, c["interleaved"]),
           "k": _norm_rotate(xk, s["wk"], cos, sin, c["interleaved"])}
    if c["train"]:
        dxq, out["dwq"] = _norm_rotate_gradient(s["dq"], xq, s["wq"], cos, sin, c["interleaved"])
        dxk, out["dwk"] = _norm_rotate_gradient(s["dk"], xk, s["wk"], cos, sin, c["interleaved"])
        out["dqk"] = torch.cat([dxq.flatten(1), dxk.flatten(1)], 1)
    return out


def _attn_plain(s, c):
    t, hq, hkv, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    g = hq // hkv
    q = s["q"].float().permute(1, 0, 2).reshape(hkv, g * t, d)      # the query heads of one key/value head together
    k, v = (s[n].float().permute(1, 0, 2).contiguous() for n in "kv")
    j = torch.arange(t, device="cuda")
    allowed = (j >= s["spans"][:, :1]) & (j < s["spans"][:, 1:])
    z = (q @ k.transpose(1, 2)).view(hkv, g, t, t).mul_(s["scale"])
    th = None
    if c["cap"]:
        th = (z / c["cap"]).tanh_()
        z = th * c["cap"]
    if s["slopes"] is not None:
        z -= s["slopes"].view(hkv, g, 1, 1) * (j[:, None] - j).abs()
    z.masked_fill_(~allowed, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)                         # a row with nothing to attend to
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).view(hq, t)
    p /= torch.where(total == 0, 1.0, total)
    o = p.view(hkv, g * t, t) @ v
    out = {"o": o.view(hq, t, d).permute(1, 0, 2).to(torch.bfloat16), "lse": lse}
    if not c["train"]:
        return out
    do = s["do"].float().permute(1, 0, 2).reshape(hkv, g * t, d)
    dv = p.view(hkv, g * t, t).transpose(1, 2) @ do
    dz = (do @ v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).view(hkv, g, t, t).mul_(p)
    if th is not None:
        dz *= th.square_().neg_().add_(1)
    dz = dz.view(hkv, g * t, t).mul_(s["scale"])
    out["dq"] = (dz @ k).view(hq, t, d).permute(1, 0, 2).to(torch.bfloat16)
    out["dk"] = (dz.transpose(1, 2) @ q).permute(1, 0, 2).to(torch.bfloat16)
    out["dv"] = dv.permute(1, 0, 2).to(torch.bfloat16)
    return out


def run(state):
    c = state["case"]
    if c["op"] == "rope":
        return (_rope_own if own else _rope_plain)(state, c)
    return (_attn_own if own else _attn_plain)(state, c)


def _pairs(case):
    """Query/key pairs that attend to one another, of one query head."""
    lo, hi = _spans(case)
    return sum(max(0, b - a) for a, b in zip(lo, hi))


def work(case):
    t, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        n = t * (hq + hkv) * d
        tables = min(t, 2048) * case["rot"] * 4 + 4 * t + 8 * d
        if not case["train"]:
            return {"bytes": 4 * n + tables, "flops": 8 * n}
        # forward: x in, y out; backward: x and dy in, dx out, both weights' gradients
        return {"bytes": 10 * n + 2 * tables + 8 * d, "flops": 26 * n}
    pairs, qn, kvn = _pairs(case), 2 * t * hq * d, 2 * t * hkv * d
    forward = 2 * qn + 2 * kvn + 4 * t * hq + 8 * t
    if not case["train"]:
        return {"bytes": forward, "flops": 4 * d * pairs * hq}
    # backward: q, k, v, o, do and lse in, dq, dk, dv out; five products
    return {"bytes": forward + 4 * qn + 4 * kvn + 4 * t * hq + 8 * t, "flops": 14 * d * pairs * hq}


def _rope_exact(s, c):
    hq, hkv, d, rot = c["q_heads"], c["kv_heads"], c["dim"], c["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.atan2(s["sin"].double(), s["cos"].double()))
    turn = turn * torch.hypot(s["sin"].double(), s["cos"].double())
    turn = turn[s["positions"].long()][:, None]                      # [tokens][1][rot / 2]
    pairs = torch.arange(rot, device="cuda").view(-1, 2) if c["interleaved"] else torch.arange(rot, device="cuda").view(2, -1).t()

    def turned(x, by):
        z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * by
        y = x.clone()
        y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z.real, z.imag
        return y

    out, dx = {}, []
    for name, first, heads in (("q", 0, hq), ("k", hq, hkv)):
        x = s["qkv"][:, first * d:(first + heads) * d].double().view(-1, heads, d)
        w = s["w" + name].double()
        norm = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        out[name] = turned(x / norm * w, turn)
        if c["train"]:
            dn = turned(s["d" + name].double(), turn.conj())
            out["dw" + name] = torch.einsum("thd,thd->d", dn, x / norm)
            along = torch.einsum("thd,thd->th", dn * w, x)[..., None]
            dx.append((dn * w / norm - x * along / (d * norm.pow(3))).flatten(1))
    if dx:
        out["dqk"] = torch.cat(dx, 1)
    return out


def _attn_exact(s, c):
    t, hq, hkv = c["tokens"], c["q_heads"], c["kv_heads"]
    at = torch.arange(t, device="cuda")
    outside = (at[None] < s["spans"][:, 0, None]) | (at[None] >= s["spans"][:, 1, None])
    names = ["o", "lse"] + (["dq", "dk", "dv"] if c["train"] else [])
    out = {n: [] for n in names}
    for h in range(hq):
        kvh = h // (hq // hkv)
        q, k, v = s["q"][:, h].double(), s["k"][:, kvh].double(), s["v"][:, kvh].double()
        x = torch.einsum("id,jd->ij", q, k) * s["scale"]
        if c["cap"]:
            x = torch.tanh(x / c["cap"])
            slope_of_cap = 1 - x * x
            x = x * c["cap"]
        if s["slopes"] is not None:
            x = x - s["slopes"][h].double() * (at[None] - at[:, None]).abs()
        x[outside] = -math.inf
        lse = torch.logsumexp(x, 1)
        p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None])
        o = p @ v
        out["o"].append(o)
        out["lse"].append(lse)
        if c["train"]:
            do = s["do"][:, h].double()
            dp = do @ v.t()
            dx = p * (dp - (p * dp).sum(1, keepdim=True))
            if c["cap"]:
                dx = dx * slope_of_cap
            dx = dx * s["scale"]
            first = h % (hq // hkv) == 0
            for n, g in (("dk", dx.t() @ q), ("dv", p.t() @ do)):
                if first:
                    out[n].append(g)
                else:
                    out[n][-1] += g
            out["dq"].append(dx @ k)
    return {n: torch.stack(x, 0 if n == "lse" else 1) for n, x in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return (_rope_exact if case["op"] == "rope" else _attn_exact)(s, case)
