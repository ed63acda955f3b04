"""Norm with rotation and window attention at the ends of their ranges: more than 2^31 elements, very many short
sequences, very many heads."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain
from tests.parity import REL_L2
from tests.test_gpu_norm_rope import DEV, freqs, rnd, weight
from tests.test_gpu_window import SCALE, backward, forward, tensors

pytestmark = pytest.mark.gpu


def test_norm_rope_past_two_to_the_31_elements():
    """One packed projection of 2.3e9 elements; the last tokens, the ones around 2^31 and the first against 64 bits, and
    the weights' gradients of a dy that is zero but for those tokens."""
    heads, N = [64, 8, 8, 8, 1], 200000
    x, f = rnd(1, N, sum(heads), 128, seed=1), freqs(64)
    assert x.numel() > 2 ** 31
    ws = [weight(1), weight(2), None, weight(3), weight(4)]
    rotate = [True, True, False, True, True]
    at = torch.cat([torch.arange(a, a + 40, device=DEV) for a in (0, 2 ** 31 // (89 * 128) - 20, N - 40)])
    dy = [torch.zeros(1, N, h, 128, dtype=torch.bfloat16, device=DEV) for h in heads]
    for i, d in enumerate(dy):
        d[:, at] = rnd(1, len(at), heads[i], 128, seed=2 + i)
    xs = x.split(heads, 2)
    ys = msa.msa_norm_rope_forward(xs, ws, f, rotate=rotate)
    dx = torch.empty_like(x)
    dxs, dws = msa.msa_norm_rope_backward(xs, ws, dy, f, rotate=rotate, dxs=dx.split(heads, 2))
    pos = at.view(1, -1)
    for i in range(5):
        want = plain.norm_rope(xs[i][:, at], ws[i], pos, f if rotate[i] else None, False, 1e-6, dy[i][:, at])
        plain.check(f"y{i}", ys[i][:, at], want["y"])
        plain.check(f"dx{i}", dxs[i][:, at], want["dx"])
        if ws[i] is not None:
            plain.check(f"dw{i}", dws[i], want["dw"])
        dxs[i][:, at] = 0
        assert not dxs[i].any()


@pytest.mark.parametrize("heads", [[1024], [1024] * 8])
def test_norm_rope_of_many_heads(heads):
    B, N = 2, 3
    x, f = rnd(B, N, sum(heads), 128, seed=20), freqs(128)
    dy = rnd(B, N, sum(heads), 128, seed=21)
    ws = [weight(i) for i in range(len(heads))]
    ys = msa.msa_norm_rope_forward(x.split(heads, 2), ws, f)
    dxs, dws = msa.msa_norm_rope_backward(x.split(heads, 2), ws, [d.contiguous() for d in dy.split(heads, 2)], f)
    pos = torch.arange(N, device=DEV).expand(B, N)
    for i, (a, d) in enumerate(zip(x.split(heads, 2), dy.split(heads, 2))):
        want = plain.norm_rope(a, ws[i], pos, f, False, 1e-6, d)
        plain.check("y", ys[i], want["y"])
        plain.check("dx", dxs[i], want["dx"])
        plain.check("dw", dws[i], want["dw"])


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", [(70000, 3, 4, 2, 2, 1), (200000, 1, 16, 1, 5, 0), (66000, 2, 8, 8, 9, 0)])
def test_window_of_many_short_sequences(B, S, Hq, Hkv, W, ns):
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=30)
    o, lse = forward(q, k, v, W, ns)
    grads = backward(q, k, v, o, lse, do, W, ns)
    want = plain.window(q, k, v, W, ns, SCALE, do)
    assert plain.check("o", o, want["o"]) <= REL_L2
    plain.check("lse", lse, want["lse"])
    for name, x in zip(("dq", "dk", "dv"), grads):
        rel = plain.check(name, x, want[name])
        assert rel <= REL_L2 or S == 1 and name != "dv"  # one key: dQ = dK = 0


@pytest.mark.parametrize("B,Hq,Hkv", [(100000, 16, 8), (20000, 128, 128)])
def test_decode_of_many_sequences(B, Hq, Hkv):
    _, k, v, _ = tensors(B, 3, 1, Hkv, seed=31)
    q = tensors(B, 1, Hq, Hkv, seed=32)[0][:, 0].contiguous()
    n = torch.arange(B, device=DEV, dtype=torch.int32) % 3 + 1
    o, lse = msa.msa_window_decode(q, k, v, n, 2, 0, SCALE)
    t = torch.arange(3, device=DEV)
    seen = (t < n[:, None]) & (t >= n[:, None] - 2)
    K, V = (x.double().repeat_interleave(Hq // Hkv, 2) for x in (k, v))
    s = torch.einsum("bhd,bjhd->bhj", q.double(), K) * SCALE
    s = s.masked_fill(~seen[:, None], -torch.inf)
    ref = s.logsumexp(-1)
    p = (s - ref[..., None]).exp()
    y = torch.einsum("bhj,bjhd->bhd", p, V)
    plain.check("o", o, (y, plain.HALF * y.abs() + (plain.HALF + plain.F) * torch.einsum("bhj,bjhd->bhd", p, V.abs())))
    plain.check("lse", lse, (ref, torch.full_like(ref, plain.F)))
