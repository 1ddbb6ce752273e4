"""Plain 64-bit forms of the attention and norm/rotation operators, with the
error bounds their tests hold the kernels to (test code, independent of the
CUDA sources; written from the formulas in include/nvfp4.h).

The bounds follow from the roundings the header names.  u = 2^-8 is bf16's
unit roundoff (8 significant bits); F = 2^-12 covers what is FP32 (scores and
statistics: a score's relative error is below 2^-20 of sum |q k|, which the
inputs here keep below 2^8, so a probability is off by less than 2^-12 of
itself).
"""
import math

import torch

U = 2.0 ** -8
F = 2.0 ** -12


def attention(q, k, v, spans, scale, softcap=0.0, slopes=None, dout=None):
    """float64 tensors [tokens, heads, dim] in, dict of results and bounds out.

    o_tol: the probabilities' rounding (u of each term), FP32 effects and the
    output's rounding.  Gradients: dS is off by what delta is off (out's own
    error times dout), by FP32 effects and by its rounding to bf16."""
    T, HQ, D = q.shape
    G = HQ // k.shape[1]
    i = torch.arange(T, device=q.device)
    lo, hi = spans[:, 0].clamp(min=0), spans[:, 1].clamp(max=T)
    ok = (i[None] >= lo[:, None]) & (i[None] < hi[:, None])
    r = {n: torch.zeros_like(q) for n in ("o", "o_tol", "dq", "dq_tol")}
    r |= {n: torch.zeros_like(k) for n in ("dk", "dk_tol", "dv", "dv_tol")}
    r["lse"] = torch.empty((HQ, T), dtype=torch.float64, device=q.device)
    for h in range(HQ):
        g = h // G
        qh, kh, vh = q[:, h], k[:, g], v[:, g]
        # rows that nothing reads may hold anything: take them out of the sums
        seen = ok.any(0)
        kh, vh = torch.where(seen[:, None], kh, 0.0), torch.where(seen[:, None], vh, 0.0)
        alive = ok.any(1)
        qh = torch.where(alive[:, None], qh, 0.0)
        z = qh @ kh.T * scale
        th = torch.tanh(z / softcap) if softcap else torch.zeros_like(z)
        s = softcap * th if softcap else z
        if slopes is not None:
            s = s - slopes[h] * (i[:, None] - i[None]).abs()
        s = s.masked_fill(~ok, -math.inf)
        lse = torch.logsumexp(s, 1)
        p = torch.where(ok, torch.exp(s - torch.where(alive, lse, 0.0)[:, None]), 0.0)
        o = p @ vh
        r["o"][:, h], r["lse"][h] = o, lse
        o_tol = (U + F) * (p @ vh.abs()) + U * o.abs()
        r["o_tol"][:, h] = o_tol
        if dout is None:
            continue
        do = torch.where(alive[:, None], dout[:, h], 0.0)
        dp = do @ vh.T
        delta = (do * o).sum(1, keepdim=True)
        damp = (1 - th * th) * scale
        dz = p * (dp - delta) * damp
        delta_tol = (do.abs() * o_tol).sum(1, keepdim=True)
        dz_tol = p * damp * (delta_tol + F * (dp.abs() + delta.abs()) + 2.0 ** -20 * (do.abs() @ vh.abs().T)) + \
            (U + F) * dz.abs() + p * scale * 2.0 ** -20 * (dp - delta).abs()
        r["dq"][:, h] = dz @ kh
        r["dq_tol"][:, h] = dz_tol @ kh.abs() + U * r["dq"][:, h].abs()
        r["dk"][:, g] += dz.T @ qh
        r["dk_tol"][:, g] += dz_tol.T @ qh.abs()
        r["dv"][:, g] += p.T @ do
        r["dv_tol"][:, g] += (U + F) * (p.T @ do.abs())
    r["dk_tol"] += U * r["dk"].abs()
    r["dv_tol"] += U * r["dv"].abs()
    return r


def rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim]; cos, sin [tokens, rot / 2]."""
    n = cos.shape[1]
    even = torch.arange(n, device=x.device) * (2 if interleaved else 1)
    odd = even + (1 if interleaved else n)
    y = x.clone()
    y[..., even] = x[..., even] * cos[:, None] - x[..., odd] * sin[:, None]
    y[..., odd] = x[..., odd] * cos[:, None] + x[..., even] * sin[:, None]
    return y


def norm_rope(x, w, cos, sin, interleaved, eps):
    return rotate(x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w, cos, sin, interleaved)


def norm_rope_backward(dy, x, w, cos, sin, interleaved, eps):
    """(dx, dw, sum of |terms| of dx, of dw)"""
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    dn = rotate(dy, cos, -sin, interleaved)
    xh, g = x * r, dn * w
    mean = (g * xh).mean(-1, keepdim=True)
    dn_abs = rotate(dy.abs(), cos.abs(), -sin.abs(), interleaved).abs() + \
        rotate(dy.abs(), cos.abs(), sin.abs(), interleaved).abs()
    size = r * (dn_abs * w.abs() + xh.abs() * (dn_abs * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return r * (g - xh * mean), (dn * xh).sum((0, 1)), size, (dn_abs * xh.abs()).sum((0, 1))
