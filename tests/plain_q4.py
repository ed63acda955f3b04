"""Plain 64-bit form of the caches in 4 bits and of attention over them.

A row x of 128: a = max |x| / 6, e = floor(log2 a) - 7 within -100 .. 90, a scale for 16 values and the codes each
rounded to the nearest member of their grid, of two equally near the one with an even last bit.

The decode steps compute with these values exactly; their roundings are those of the softmax weights to fp16 (HALF16, and
2^-25 of the largest weight below fp16's normal range) and of o to bf16, and fp32 arithmetic (F, as in plain_local).
"""
import torch

from tests.plain_local import F, HALF

HALF16 = torch.finfo(torch.float16).eps / 2
CODES = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
SCALES = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** p for p in range(-6, 9) for m in range(8)][:119]


def nearest(v, grid):
    """Place in the ascending grid of the member nearest to v >= 0."""
    g = torch.tensor(grid, dtype=torch.float64, device=v.device)
    i = torch.searchsorted(g, v.contiguous()).clamp(1, len(grid) - 1)
    below, above = v - g[i - 1], g[i] - v
    return torch.where((below < above) | ((below == above) & (i % 2 == 1)), i - 1, i)


def quantise(x):
    """bf16 rows [..., 128] -> (codes [..., 128], scale bytes [..., 8], exponent bytes [...]) as int64."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0)
    a = x.abs().amax(-1) / 6
    e = torch.where(a > 0, torch.frexp(a).exponent.double() - 8, -100).clamp(-100, 90)  # (a logarithm may miss a power of two)
    e = torch.where(finite, e, 0)
    y = (x * torch.exp2(-e)[..., None]).unflatten(-1, (8, 16))
    s = nearest(y.abs().amax(-1) / 6, SCALES)
    f = torch.tensor(SCALES, dtype=torch.float64, device=x.device)[s][..., None]
    c = nearest(torch.where(f > 0, y.abs() / f, 0), CODES)
    c = c + 8 * ((y < 0) & (c > 0))
    s = torch.where(finite[..., None], s, 0x7f)
    return c.flatten(-2), s, (e + 127).long()


def values(parts):
    """fp64 values of (codes, scales, exponents); NaN where the scale is."""
    c, s, e = parts
    grid = torch.tensor(CODES + [-x for x in CODES], dtype=torch.float64, device=c.device)
    scale = torch.tensor(SCALES + [float("nan")], dtype=torch.float64, device=c.device)[s & 127]
    x = grid[c].unflatten(-1, (8, 16)) * scale[..., None] * torch.exp2(e.double() - 127)[..., None, None]
    return x.flatten(-2)


def unpack(cache):
    """uint8 [B, H, blocks, 9344] -> (codes [B, rows, H, 128], scales, exponents) as int64."""
    b = cache.long()
    data, s, e = b[..., :8192].unflatten(-1, (128, 64)), b[..., 8192:9216].unflatten(-1, (128, 8)), b[..., 9216:]
    c = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    rows = lambda x: x.flatten(2, 3).transpose(1, 2)  # noqa: E731
    return rows(c), rows(s), e.flatten(2, 3).transpose(1, 2)


def attend(q, k, v, scale):
    """One sequence: q [Hq, 128], k, v [n, Hkv, 128] fp64 -> {o, lse} with bounds."""
    Hq, n = q.shape[0], k.shape[0]
    K, V = (x.transpose(0, 1).repeat_interleave(Hq // x.shape[1], 0) for x in (k, v))
    s = (K @ q.double().unsqueeze(-1)).squeeze(-1) * scale
    lse = s.logsumexp(-1)
    p = (s - lse[:, None]).exp().unsqueeze(1)
    o = (p @ V).squeeze(1)
    # a row's largest kept value is at most 1536 of its power of two, and at least half of that
    small = n * 2.0 ** -25 * 2 * V.abs().amax((1, 2), keepdim=True).squeeze(-1)
    return {"o": (o, HALF * o.abs() + (HALF16 + F) * (p @ V.abs()).squeeze(1) + small), "lse": (lse, torch.full_like(lse, F))}


def window_keys(n, window, sinks, device):
    j = torch.arange(n, device=device)
    return j[(j >= n - window) | (j < sinks)]
