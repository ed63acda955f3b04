"""Plain 64-bit implementations of the window attention and of the norm with rotation, with element-wise
error bounds for results computed from bf16 inputs with fp32 sums.

HALF is the largest relative error of one rounding to bf16 (half a step).  A bound counts the
roundings to bf16 that the operators make -- of an output, of P and of dS before their products, of
the stored O that D is taken from -- at their worst, and gives fp32 arithmetic a relative share F.
F covers: scores as sums of 128 exact products (at most 128 * 2^-24 of sum |q k| scale, about 7 for
normal inputs: 5.5e-5 absolute in the exponent, hence relative in P), the same again through the LSE,
and exponentials and sums (2^-21).
"""
import torch

HALF = torch.finfo(torch.bfloat16).eps / 2
F = 2e-4


def visible(S, window, sinks, device="cpu"):
    t = torch.arange(S, device=device)
    d = t[:, None] - t
    return (d >= 0) & ((d < window) | (t < sinks))


def _heads(x, n):  # [B, S, h, D] -> [B, n, S, D] fp64
    x = x.double().transpose(1, 2)
    return x.repeat_interleave(n // x.shape[1], 1)


def window(q, k, v, window_, sinks, scale, dout=None):
    """{name: (value, bound)} of o, lse and, with dout, dq, dk, dv."""
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    Q, K, V = _heads(q, Hq), _heads(k, Hq), _heads(v, Hq)
    seen = visible(S, window_, sinks, q.device)
    s = (Q @ K.transpose(-1, -2) * scale).masked_fill(~seen, -torch.inf)
    lse = s.logsumexp(-1)
    p = (s - lse[..., None]).exp()
    o = p @ V
    eo = HALF * o.abs() + (HALF + F) * (p @ V.abs())
    back = lambda x: x.transpose(1, 2)  # noqa: E731
    group = lambda x: x.view(B, Hkv, Hq // Hkv, S, D).sum(2).transpose(1, 2)  # noqa: E731
    out = {"o": (back(o), back(eo)), "lse": (lse, torch.full_like(lse, F))}
    if dout is None:
        return out
    G = _heads(dout, Hq)
    dp = G @ V.transpose(-1, -2)
    dd = (G * o).sum(-1, keepdim=True)
    ed = (G.abs() * eo).sum(-1, keepdim=True)
    ds = scale * p * (dp - dd)
    es = HALF * ds.abs() + scale * p * (F * (dp.abs() + dd.abs()) + ed * (1 + HALF))
    dq, eq = ds @ K, es @ K.abs()
    dk, ek = group(ds.transpose(-1, -2) @ Q), group(es.transpose(-1, -2) @ Q.abs())
    dv = group(p.transpose(-1, -2) @ G)
    ev = group((HALF + F) * (p.transpose(-1, -2) @ G.abs()))
    out["dq"] = (back(dq), back(eq + HALF * (dq.abs() + eq)))
    out["dk"] = (dk, ek + HALF * (dk.abs() + ek))
    out["dv"] = (dv, ev + HALF * (dv.abs() + ev))
    return out


def window_decode(q, k, v, lens, window_, sinks, scale):
    """Rows of o [B, Hq, D], lse [B, Hq] with bounds, one sequence at a time over its visible rows."""
    B, Hq, D = q.shape
    Hkv = k.shape[2]
    vals = [], [], []
    for b, n in enumerate(lens):
        j = torch.arange(n, device=k.device)
        j = j[(j >= n - window_) | (j < sinks)]
        K = k[b, j].double().transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
        V = v[b, j].double().transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
        s = (K @ q[b].double().unsqueeze(-1)).squeeze(-1) * scale
        lse = s.logsumexp(-1)
        p = (s - lse[:, None]).exp().unsqueeze(1)
        o = (p @ V).squeeze(1)
        vals[0].append(o)
        vals[1].append(HALF * o.abs() + (HALF + F) * (p @ V.abs()).squeeze(1))
        vals[2].append(lse)
    o, eo, lse = (torch.stack(x) for x in vals)
    return {"o": (o, eo), "lse": (lse, torch.full_like(lse, F))}


def check(name, got, want):
    """got within the bound of want everywhere; prints the worst share of the bound."""
    value, bound = want
    got = got.detach().double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} values not finite"
    err = (got - value).abs()
    bad = err > bound + 1e-30
    if bad.any():
        at = [int(i) for i in bad.nonzero()[0]]
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values over their bound; first at {at}: "
                             f"{float(got[tuple(at)])} for {float(value[tuple(at)])}, bound {float(bound[tuple(at)]):.2e}")
    norm = float(value.norm())
    rel = float(err.norm()) / norm if norm else 0.0
    return rel


# ------------------------------------------------------------------------------------ norm, rotation
# fp32 share: mean of squares (a tree over 128), rsqrt, three products, and the rotation with an angle
# exact to 2^-32 turns rounded to fp32 (4e-7): together under 3e-6 of the two elements of a pair.
FR = 4e-6


def rotate(u, positions, inv_freq, interleaved, sign=1):
    """u [B, N, H, 128] fp64 turned by sign * position * inv_freq, a pair at a time."""
    if inv_freq is None:
        return u
    y = u.clone()
    half = inv_freq.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = sign * positions.double() * float(inv_freq[i])
        c, s = ang.cos()[..., None], ang.sin()[..., None]
        y[..., a] = u[..., a] * c - u[..., b] * s
        y[..., b] = u[..., b] * c + u[..., a] * s
    return y


def pair_sum(u, inv_freq, interleaved):
    """|u| of an element and its partner: what an error of the rotation is relative to."""
    u = u.abs()
    if inv_freq is None:
        return u
    half, y = inv_freq.numel(), u.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = y[..., b] = u[..., a] + u[..., b]
    return y


def norm_rope(x, w, positions, inv_freq, interleaved, eps, dy=None):
    """{name: (value, bound)} of y and, with dy, dx and (where w) dw."""
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    u = x if w is None else w.double() * x * r
    y = rotate(u, positions, inv_freq, interleaved)
    out = {"y": (y, HALF * y.abs() + FR * pair_sum(u, inv_freq, interleaved))}
    if dy is None:
        return out
    dy = dy.double()
    g, eg = rotate(dy, positions, inv_freq, interleaved, -1), FR * pair_sum(dy, inv_freq, interleaved)
    if w is None:
        out["dx"] = (g, HALF * g.abs() + eg)
        return out
    h, w = g * w.double(), w.double()
    m = (h * x).mean(-1, keepdim=True)
    dx = r * h - x * r ** 3 * m
    size = r * (h.abs() + eg / FR * w.abs()) + x.abs() * r ** 3 * ((h.abs() + eg / FR * w.abs()) * x.abs()).mean(-1, keepdim=True)
    out["dx"] = (dx, HALF * dx.abs() + 2 * FR * size)
    # sums of fp32 terms in short runs: 64 rows of a warp's token, at most some hundred tokens, blocks in fp64
    out["dw"] = ((g * x * r).sum((0, 1, 2)), (1e-5 * ((g.abs() + eg / FR) * x.abs() * r)).sum((0, 1, 2)))
    return out
