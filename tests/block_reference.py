"""Plain 64-bit forms of the operators of a block's feed-forward half, written
from their formulas, with the sizes of the terms that bounds are made of."""
import torch


def checkpoint(x):
    """(values, scale bytes) of a matrix kept in 8 bits: E4M3 codes times a power of two per 1x32 block."""
    x = x.double()
    rows, cols = x.shape
    blocks = -(-cols // 32)
    pad = torch.zeros(rows, blocks * 32, dtype=torch.float64, device=x.device)
    pad[:, :cols] = torch.where(torch.isfinite(x), x, 0.0)
    amax = pad.view(rows, blocks, 32).abs().amax(-1)
    # the smallest power of two with amax <= 448 of it: amax = m 2^k, 1/2 <= m < 1, 448 = 0.875 2^9
    m, k = torch.frexp(amax)
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(amax == 0, torch.full_like(e, -117), e).clamp(min=-117)
    scale = torch.exp2(e.double()).repeat_interleave(32, 1)[:, :cols]
    v = torch.where(torch.isfinite(x), x, 0.0) / scale
    step = torch.exp2((torch.frexp(v)[1].double() - 4).clamp(min=-9))
    v = torch.round(v / step) * step
    v = torch.where(scale == 2.0 ** 120, v.clamp(-240, 240), v) * scale   # 2^128 is no FP32 number
    return torch.where(torch.isfinite(x), v, float("nan")), (e + 127).to(torch.uint8)


def over(x, eps):
    """1 / sqrt(mean(x^2) + eps) per row."""
    return (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def block_norm(r, y, post, gate, scale, eps):
    """(r', the size of its terms)."""
    if y is None:
        return scale * r, (scale * r).abs()
    h = y if post is None else y * over(y, eps) * post
    gh = h if gate is None else gate * h
    return scale * r + gh, (scale * r).abs() + gh.abs()


def block_norm_backward(dr, dn, x, y, post, pre, gate, scale, eps):
    """{name: (gradient, size of its terms)} from the formulas of the operator."""
    zero = torch.zeros_like(x)
    d, dsize = (zero if dr is None else dr), (zero if dr is None else dr.abs())
    out = {}
    if pre is not None:
        rq = over(x, eps)
        xh, g = x * rq, dn * pre
        d = d + rq * (g - xh * (g * xh).mean(-1, keepdim=True))
        dsize = dsize + rq * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
        out["dpre_weight"] = (dn * xh).sum(0), (dn * xh).abs().sum(0)
    out["dresidual"] = scale * d, abs(scale) * dsize
    if y is None:
        return out
    rp = over(y, eps) if post is not None else torch.ones_like(y[:, :1])
    a = y * rp
    h = a if post is None else a * post
    c = torch.ones_like(y) if gate is None else gate.expand_as(y)
    if gate is not None:
        dg, gs = d * h, dsize * h.abs()
        out["dgate"] = (dg.sum(0), gs.sum(0)) if gate.dim() == 1 else (dg, gs)
    t, ts = d * c, dsize * c.abs()
    if post is None:
        out["dbranch"] = t, ts
        return out
    out["dpost_weight"] = (t * a).sum(0), (ts * a.abs()).sum(0)
    t, ts = t * post, ts * post.abs()
    out["dbranch"] = (rp * (t - a * (t * a).mean(-1, keepdim=True)),
                      rp * (ts + a.abs() * (ts * a.abs()).mean(-1, keepdim=True)))
    return out
