"""Window attention on tensors of more than 2^31 elements, every row of one KV head's group against 64 bits, and dV of
windows so short that dQ and dK vanish."""
import pytest
import torch

from tests import plain_local as plain
from tests.parity import REL_L2
from tests.test_gpu_window import CASES, DEV, SCALE, backward, forward, tensors

pytestmark = pytest.mark.gpu


def group_reference(q, k, v, do, g, W, ns):
    """{name: (value, bound)} of the last sequence's KV head g and its query heads, with the bounds of plain_local.window:
    a chunk of queries against the sinks and the window's keys, gathered."""
    S, Hkv = k.shape[1:3]
    G = q.shape[2] // Hkv
    hs = slice(g * G, g * G + G)
    q, k, v, do = (x[-1] for x in (q, k, v, do))
    new = lambda *n: torch.zeros(n, dtype=torch.float64, device=DEV)  # noqa: E731
    val = dict(o=new(S, G, 128), lse=new(S, G), dq=new(S, G, 128), dk=new(S, 128), dv=new(S, 128))
    err = {n: torch.zeros_like(x) for n, x in val.items()}
    H, F = plain.HALF, plain.F
    for a in range(0, S, 2048):
        t = torch.arange(a, min(S, a + 2048), device=DEV)
        j = torch.cat([torch.arange(ns, device=DEV).expand(len(t), ns), t[:, None] - W + 1 + torch.arange(W, device=DEV)], 1)
        near = torch.arange(ns + W, device=DEV) >= ns
        seen = (j >= 0) & (j <= t[:, None]) & (near | (j <= t[:, None] - W))
        j = j.clamp(0, S - 1)
        Q, O = q[t, hs].double(), do[t, hs].double()
        K, V = k[j, g].double(), v[j, g].double()
        s = torch.einsum("tgd,tjd->tgj", Q, K).mul_(SCALE).masked_fill_(~seen[:, None], -torch.inf)
        lse = s.logsumexp(-1)
        p = (s - lse[..., None]).exp()
        o = torch.einsum("tgj,tjd->tgd", p, V)
        eo = H * o.abs() + (H + F) * torch.einsum("tgj,tjd->tgd", p, V.abs())
        dp = torch.einsum("tgd,tjd->tgj", O, V)
        dd, ed = (O * o).sum(-1, keepdim=True), (O.abs() * eo).sum(-1, keepdim=True)
        ds = SCALE * p * (dp - dd)
        es = H * ds.abs() + SCALE * p * (F * (dp.abs() + dd.abs()) + ed * (1 + H))
        for name, x, e in (("o", o, eo), ("lse", lse, torch.full_like(lse, F)),
                           ("dq", torch.einsum("tgj,tjd->tgd", ds, K), torch.einsum("tgj,tjd->tgd", es, K.abs()))):
            val[name][t], err[name][t] = x, e
        at = j.flatten()
        for name, x, e, rows in (("dk", ds, es, Q), ("dv", p, (H + F) * p, O)):
            val[name].index_add_(0, at, torch.einsum("tgj,tgd->tjd", x, rows).flatten(0, 1))
            err[name].index_add_(0, at, torch.einsum("tgj,tgd->tjd", e, rows.abs()).flatten(0, 1))
    for name in ("dq", "dk", "dv"):
        err[name] += H * (val[name].abs() + err[name])
    return {n: (val[n], err[n]) for n in val}


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", [
    (1, 270000, 64, 8, 140, 4),   # 2.2e9 elements of q: two key tiles a unit, one long list for the sinks' block
    (1, 270000, 64, 8, 40, 130),  # sinks past a key block: two long lists
    (5, 60000, 64, 64, 20, 1),    # K and V of 2.4e9 elements, one head a group
])
def test_past_two_to_the_31_elements(B, S, Hq, Hkv, W, ns):
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=60)
    assert q.numel() > 2 ** 31
    o, lse = forward(q, k, v, W, ns)
    dq, dk, dv = backward(q, k, v, o, lse, do, W, ns)
    G = Hq // Hkv
    for g in (0, Hkv - 1):
        want = group_reference(q, k, v, do, g, W, ns)
        hs = slice(g * G, g * G + G)
        for name, x in (("o", o[-1, :, hs]), ("lse", lse[-1, hs].T), ("dq", dq[-1, :, hs]), ("dk", dk[-1, :, g]),
                        ("dv", dv[-1, :, g])):
            rel = plain.check(name, x, want[name])
            assert rel <= REL_L2, (name, rel)


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", [c for c in CASES if min(c[1], c[4]) <= 2])
def test_dv_of_the_shortest_windows(B, S, Hq, Hkv, W, ns):
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=S + W)
    o, lse = forward(q, k, v, W, ns)
    dv = backward(q, k, v, o, lse, do, W, ns)[2]
    assert plain.check("dv", dv, plain.window(q, k, v, W, ns, SCALE, do)["dv"]) <= REL_L2
