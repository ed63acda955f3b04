"""Norm and rotation by positions of several axes: against the one-axis operator and a plain 64-bit form."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain
from tests import plain_q4
from tests.plain_local import check
from tests.test_gpu_q4 import same_rows

pytestmark = pytest.mark.gpu


def make(seed, B, N, heads, rot, A):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((B, N, sum(heads), 128), generator=g, device="cuda").to(torch.bfloat16)
    ws = [1 + 0.1 * torch.randn(128, generator=g, device="cuda") for _ in heads]
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (A, B, N), generator=g, device="cuda").to(torch.int32)
    pos[:, :, 1:] = torch.randint(0, 5000, (A, B, N - 1), generator=g, device="cuda").to(torch.int32)
    dy = [torch.randn((B, N, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in heads]
    return x, ws, freq, pos, dy


def rotate(u, pos, freq, axes, inter, sign=1):
    """u fp64, a pair at a time by its axis's positions."""
    y, half = u.clone(), freq.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        # whole turns taken off in exact arithmetic where the product has more than 53 bits: int32 x fp32 has 55
        ang = sign * pos[axes[i]].double() * float(freq[i])
        c, s = ang.cos()[..., None], ang.sin()[..., None]
        y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    return y


def plain_axes(x, w, pos, freq, axes, inter, dy=None):
    """plain_local.norm_rope with the rotation above."""
    old, turn = plain.rotate, lambda u, p, f, i, sign=1: rotate(u, pos, freq, axes, inter, sign)
    plain.rotate = turn
    try:
        return plain.norm_rope(x, w, None, freq, inter, 1e-6, dy)
    finally:
        plain.rotate = old


@pytest.mark.parametrize("B,N,heads,rot,A,inter", [
    (1, 1, [1], 16, 1, False), (1, 1, [4, 1], 128, 3, False), (2, 3, [8, 2, 2], 64, 3, True), (1, 130, [16, 2], 128, 4, False),
    (3, 77, [5], 48, 2, True), (2, 500, [8, 2, 2, 2, 1], 96, 3, False), (1, 257, [2], 16, 4, True),
])
def test_forward_and_gradients(B, N, heads, rot, A, inter):
    x, ws, freq, pos, dy = make(rot + A, B, N, heads, rot, A)
    axes = [(7 * i + i // 3) % A for i in range(rot // 2)]
    axes[-1] = A - 1
    xs = x.split(heads, 2)
    how = dict(positions=pos, axes=axes, interleaved=inter)
    ys = msa.msa_norm_rope_forward(xs, ws, freq, **how)
    dxs, dws = msa.msa_norm_rope_backward(xs, ws, dy, freq, **how)
    for i in range(len(heads)):
        want = plain_axes(xs[i], ws[i], pos, freq, axes, inter, dy[i])
        check(f"y[{i}]", ys[i], want["y"])
        check(f"dx[{i}]", dxs[i], want["dx"])
        check(f"dw[{i}]", dws[i], want["dw"])


@pytest.mark.parametrize("inter", [False, True])
def test_one_axis_is_the_plain_rotation(inter):
    """Axes that all point to the same positions are the operator without axes."""
    x, ws, freq, pos, dy = make(3, 2, 300, [4, 2], 128, 1)
    pos3 = pos.expand(3, -1, -1).contiguous()
    xs = x.split([4, 2], 2)
    a = msa.msa_norm_rope_forward(xs, ws, freq, pos[0].contiguous(), interleaved=inter)
    b = msa.msa_norm_rope_forward(xs, ws, freq, pos3, interleaved=inter, axes=[i % 3 for i in range(64)])
    for u, v in zip(a, b):  # the same up to the contraction of a product and a sum
        assert ((u.float() - v.float()).abs() <= 2.0 ** -7 * u.float().abs() + 1e-5).all()


def test_autograd():
    x, ws, freq, pos, dy = make(5, 2, 40, [4, 1], 64, 3)
    axes = [0] * 8 + [1] * 12 + [2] * 12
    p = x.detach().requires_grad_()
    w = [t.clone().requires_grad_() for t in ws]
    ys = msa.msa_norm_rope_packed_func(p, [4, 1], w, freq, pos, axes=axes)
    torch.autograd.backward(ys, dy)
    got = torch.split(p.grad, [4, 1], 2)
    for i, part in enumerate(x.split([4, 1], 2)):
        want = plain_axes(part, ws[i], pos, freq, axes, False, dy[i])
        check("dx", got[i], want["dx"])
        check("dw", w[i].grad, want["dw"])
    a, b = (t.contiguous().requires_grad_() for t in x.split([4, 1], 2))
    ys = msa.msa_norm_rope_func([a, b], w, freq, pos, axes=axes)
    torch.autograd.backward(ys, dy)
    assert torch.equal(a.grad, got[0]) and torch.equal(b.grad, got[1])


def test_gradient_is_that_of_differences():
    """Along a random direction, in steps large enough for bf16 inputs to hold them."""
    x, ws, freq, pos, dy = make(6, 1, 64, [2], 128, 3)
    axes = [i % 3 for i in range(64)]
    d = torch.randn(x.shape, device="cuda").to(torch.bfloat16).double()
    x = x.double()
    dx, _ = msa.msa_norm_rope_backward([x.to(torch.bfloat16)], ws, dy, freq, positions=pos, axes=axes)
    f = lambda u: (plain_axes(u, ws[0], pos, freq, axes, False)["y"][0] * dy[0].double()).sum()  # noqa: E731
    h = 1e-5
    want = (f(x + h * d) - f(x - h * d)) / (2 * h)
    got = (dx[0].double() * d).sum()
    # dx is rounded to bf16: at most HALF of each term, and the difference's own error h^2
    assert abs(got - want) <= plain.HALF * (dx[0].double() * d).abs().sum() + 1e-4


@pytest.mark.parametrize("axes,A", [(None, 1), ([0] * 16 + [1] * 24 + [2] * 24, 3)])
def test_append_with_positions_of_its_own(axes, A):
    """The tokens turn by their positions and go to the rows that the lengths say."""
    B, N, cap = 3, 2, 128
    x, ws, freq, pos, _ = make(7, B, N, [4, 2, 2], 128, A)
    cache = torch.full((B, cap, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    quant = msa.msa_q4_cache(B, 2, cap, "cuda")
    xs = x.split([4, 2, 2], 2)
    n = torch.tensor([2, 77, 128], dtype=torch.int32, device="cuda")
    p = pos if axes else pos[0].contiguous()
    y, _, _ = msa.msa_norm_rope_append(xs, ws, freq, n, [None, cache, quant], positions=p, axes=axes)
    each = axes or [0] * 64
    want = [plain_axes(xs[i], ws[i], pos, freq, each, False)["y"] for i in range(3)]
    check("q", y, want[0])
    at = torch.stack([torch.arange(m - N, m) for m in n.tolist()]).cuda()
    b = torch.arange(B, device="cuda")[:, None]
    check("k", cache[b, at], want[1])
    rest = torch.ones(B, cap, dtype=torch.bool, device="cuda")
    rest[b, at] = False
    assert (cache[rest] == 3).all()
    assert (quant != 0).any()


def test_more_positions_than_axes_used():
    """A third axis that no pair uses may be there, with anything in it."""
    x, ws, freq, pos, _ = make(8, 1, 20, [2], 32, 3)
    axes = [0] * 8 + [1] * 8
    a = msa.msa_norm_rope_forward([x], ws, freq, positions=pos, axes=axes)
    b = msa.msa_norm_rope_forward([x], ws, freq, positions=pos[:2].contiguous(), axes=axes)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,A", [(None, 1), ([0] * 16 + [1] * 24 + [2] * 24, 3), ([i % 4 for i in range(16)], 4)])
@pytest.mark.parametrize("N,lens", [(1, [1, 77, 128]), (5, [5, 200, 256])])
def test_append_with_positions_of_its_own_in_4_bits(axes, A, interleaved, N, lens):
    """A cache in 4 bits takes what a bf16 output of the same call holds for the same rows: normed, turned by the given positions
    and rounded; at the rows that the lengths say, and no others."""
    B, cap, H = 3, 256, 3
    rot = 2 * len(axes) if axes else 128
    x, ws, freq, pos, _ = make(9 + N, B, N, [H, H], rot, A)
    k, k2 = x.split([H, H], 2)
    k2.copy_(k)
    ws = [ws[0], ws[0]]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = msa.msa_q4_cache(B, H, cap, "cuda")
    p = pos if axes else pos[0].contiguous()
    state = torch.empty(256, dtype=torch.uint8, device="cuda")
    _, y = msa.msa_norm_rope_append([k, k2], ws, freq, n, [cache, None], positions=p, axes=axes, interleaved=interleaved, ws=state)
    assert msa.msa_device_status(state) == 0
    check("k", y, plain_axes(k, ws[0], pos, freq, axes or [0] * (rot // 2), interleaved)["y"])
    rows = [torch.arange(m - N, m, device="cuda") for m in lens]
    same_rows(cache, rows, y)
    for part in plain_q4.unpack(cache):
        for b in range(B):
            part[b, rows[b]] = 0
        assert not part.any()
