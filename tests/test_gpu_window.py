"""Sliding-window attention with sinks against a plain 64-bit implementation: sizes, heads and masks where
tiles begin and end, gradients against the formula and against differences, the decode step with
whatever a cache holds outside the window, repeatability, streams and captured graphs."""
import ctypes

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain
from tests.parity import REL_L2

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 128 ** -0.5


def tensors(B, S, Hq, Hkv, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda h: torch.randn((B, S, h, 128), generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    return r(Hq), r(Hkv), r(Hkv), r(Hq)


def forward(q, k, v, W, ns, scale=SCALE):
    shape = msa.make_window_shape(q, k, W, ns, scale)
    ws = msa.window_workspace(shape, msa.OP_WINDOW_FORWARD, DEV)
    o, lse = msa.msa_window_forward(q, k, v, W, ns, scale, ws=ws)
    assert msa.msa_device_status(ws) == 0
    return o, lse


def backward(q, k, v, o, lse, do, W, ns, scale=SCALE):
    shape = msa.make_window_shape(q, k, W, ns, scale)
    ws = msa.window_workspace(shape, msa.OP_WINDOW_BACKWARD, DEV)
    grads = msa.msa_window_backward(q, k, v, o, lse, do, W, ns, scale, ws=ws)
    assert msa.msa_device_status(ws) == 0
    return grads


# (B, S, Hq, Hkv, window, sinks)
CASES = [
    (1, 1, 1, 1, 1, 0),            # one token
    (2, 1, 8, 2, 5, 3),
    (1, 2, 4, 4, 1, 0),            # every query sees itself alone
    (3, 7, 16, 1, 3, 2),           # less than a tile
    (1, 127, 4, 2, 128, 0),        # just under a key block, window beyond it
    (1, 128, 8, 1, 64, 4),
    (2, 129, 2, 1, 17, 1),         # one token past a block, two sequences
    (1, 300, 8, 8, 128, 8),        # one head per group, sinks a multiple of eight
    (1, 513, 32, 2, 100, 130),     # sinks past a key block: whole and shared sink tiles
    (1, 900, 16, 1, 40, 128),      # sinks a whole block
    (2, 777, 16, 2, 256, 16),
    (1, 1000, 4, 1, 1000, 0),      # dense
    (1, 640, 8, 2, 2 ** 31 - 1, 4),  # dense, whatever the sinks
    (1, 1500, 16, 16, 33, 5),
    (1, 2100, 8, 1, 700, 257),
    (1, 260, 4, 2, 8, 300),        # more sinks than tokens
    (1, 450, 8, 4, 449, 1),        # one key short of dense
    (4, 1024, 64, 8, 200, 4),      # more units than SMs: two tiles a unit
    (1, 6000, 16, 2, 1, 1),        # windows of one key and one sink
]


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", CASES)
def test_forward(B, S, Hq, Hkv, W, ns):
    q, k, v, _ = tensors(B, S, Hq, Hkv, seed=S + W)
    o, lse = forward(q, k, v, W, ns)
    want = plain.window(q, k, v, W, ns, SCALE)
    assert plain.check("o", o, want["o"]) <= REL_L2
    plain.check("lse", lse, want["lse"])


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", CASES)
def test_backward(B, S, Hq, Hkv, W, ns):
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=S + W)
    o, lse = forward(q, k, v, W, ns)
    grads = backward(q, k, v, o, lse, do, W, ns)
    want = plain.window(q, k, v, W, ns, SCALE, do)
    for name, got in zip(("dq", "dk", "dv"), grads):
        rel = plain.check(name, got, want[name])
        # queries that see one key have dq = dk = 0: only the element-wise bound says something there
        assert rel <= REL_L2 or min(S, W) <= 2, (name, rel)


@pytest.mark.parametrize("W,ns,S", [(2, 0, 300), (3, 1, 300), (8, 0, 300), (5, 3, 300), (7, 1, 129), (900, 0, 8)])
def test_backward_of_a_few_keys(W, ns, S):
    """Rows of a few keys: D from P and dP instead of the rounded O.  What is left are the roundings of dS and of
    the result (dV: of P and of the result), each uniform within half a step of 2^-8 at worst and so at most
    2^-8 / sqrt(3) in the root mean square: 2^-8 sqrt(2 / 3) = 3.2e-3 together (2.4e-3 over all mantissas)."""
    q, k, v, do = tensors(2, S, 8, 2, seed=40)
    o, lse = forward(q, k, v, W, ns)
    want = plain.window(q, k, v, W, ns, SCALE, do)
    for name, got in zip(("dq", "dk", "dv"), backward(q, k, v, o, lse, do, W, ns)):
        assert plain.check(name, got, want[name]) <= 2 ** -8 * (2 / 3) ** 0.5


@pytest.mark.parametrize("B,S,Hq,Hkv,W,ns", [
    (2, 600, 16, 2, 12, 0), (2, 600, 8, 4, 12, 0), (2, 600, 4, 4, 12, 0), (1, 700, 16, 1, 20, 4), (1, 700, 4, 4, 20, 4),
    (2, 500, 8, 2, 2, 1), (2, 500, 4, 4, 3, 0), (16, 16, 16, 2, 256, 0), (4, 32, 32, 8, 4096, 4), (16, 24, 4, 2, 9, 30),
    (3, 333, 8, 4, 31, 1), (1, 400, 4, 4, 31, 1)])
def test_backward_of_up_to_32_keys(B, S, Hq, Hkv, W, ns):
    """Where no row sees more than 32 keys, dQ and dK carry the roundings of dS and of the result and no more: their
    relative error is that of these two done in 64 bits.  A D from the stored O adds a factor of sqrt(1 + 2.7 / n) at n
    keys, 1.04 at 32 and 1.10 at 12.  The same inputs round the same way but where fp32 moves a value across a
    boundary: with a D off by 2^-18 of itself the error differs by at most 0.3 percent, so 2 percent tell the two apart."""
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=41)
    o, lse = forward(q, k, v, W, ns)
    got = dict(zip(("dq", "dk"), backward(q, k, v, o, lse, do, W, ns)))
    Q, K, V, G = (plain._heads(x, Hq) for x in (q, k, v, do))
    s = (Q @ K.transpose(-1, -2) * SCALE).masked_fill(~plain.visible(S, W, ns, DEV), -torch.inf)
    p, dp = s.softmax(-1), G @ V.transpose(-1, -2)
    ds = SCALE * p * (dp - (p * dp).sum(-1, keepdim=True))
    group = lambda x: x.view(B, Hkv, Hq // Hkv, S, 128).sum(2).transpose(1, 2)  # noqa: E731
    once = lambda x: x.to(torch.bfloat16).double()  # noqa: E731
    want = {"dq": (ds @ K).transpose(1, 2), "dk": group(ds.transpose(-1, -2) @ Q)}
    least = {"dq": once((once(ds) @ K).transpose(1, 2)), "dk": once(group(once(ds).transpose(-1, -2) @ Q))}
    for name, ref in want.items():
        err, floor = (float((x.double() - ref).norm() / ref.norm()) for x in (got[name], least[name]))
        assert err <= 1.02 * floor, (name, err, floor)


def test_backward_of_small_runs_after_large_ones():
    """Units of one key tile leave columns of tensor memory unwritten, here behind what other launches on the same SMs
    left there: large finite scores and then NaN gradients."""
    q, k, v, do = tensors(2, 700, 16, 2, seed=42)
    o, lse = forward(q, k, v, 20, 4)
    want = backward(q, k, v, o, lse, do, 20, 4)
    big = tensors(4, 2048, 16, 2, seed=43)
    ob, lb = forward(*big[:3], 1000, 4)
    msa.msa_window_backward(*big[:3], ob, lb, torch.full_like(big[3], float("nan")), 1000, 4, SCALE)
    again = backward(q, k, v, o, lse, do, 20, 4)
    assert all(torch.isfinite(g).all() and torch.equal(a, g) for a, g in zip(want, again))


@pytest.mark.parametrize("scale,size", [(1.0, 1.0), (0.02, 3.0)])
def test_sharp_and_flat_softmax(scale, size):
    """Scores up to about +-60 (the running maximum moves, rows are rescaled) and nearly uniform ones."""
    q, k, v, do = tensors(1, 700, 8, 2, seed=5)
    q = q * size
    o, lse = forward(q, k, v, 150, 9, scale)
    s = (q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max() * scale).item()
    # the scores' fp32 sums: 128 terms of at most s in all; the exponent's error grows with them
    f = max(plain.F, 4 * 128 * 2 ** -24 * s)
    old, plain.F = plain.F, f
    try:
        want = plain.window(q, k, v, 150, 9, scale, do)
    finally:
        plain.F = old
    plain.check("o", o, want["o"])
    plain.check("lse", lse, want["lse"])
    for name, got in zip(("dq", "dk", "dv"), backward(q, k, v, o, lse, do, 150, 9, scale)):
        plain.check(name, got, want[name])


def test_rising_scores_rescale_every_tile():
    """Keys that grow along the sequence: each later tile's maximum passes the slack, so O is rescaled at
    every tile of a unit."""
    q, k, v, do = tensors(1, 1200, 4, 1, seed=6)
    k = (k.float() * torch.linspace(0.1, 4, 1200, device=DEV)[None, :, None, None]).to(torch.bfloat16)
    q = (q.float().abs()).to(torch.bfloat16)
    k = (k.float().abs()).to(torch.bfloat16)
    o, lse = forward(q, k, v, 900, 3)
    s = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * SCALE
    old, plain.F = plain.F, max(plain.F, 4 * 128 * 2 ** -24 * s)
    try:
        want = plain.window(q, k, v, 900, 3, SCALE, do)
    finally:
        plain.F = old
    plain.check("o", o, want["o"])
    plain.check("lse", lse, want["lse"])
    for name, got in zip(("dq", "dk", "dv"), backward(q, k, v, o, lse, do, 900, 3)):
        plain.check(name, got, want[name])


def test_differences():
    """<gradient, d> against central differences of sum(o * dout) in 64 bits along random directions."""
    W, ns = 50, 6
    q, k, v, do = tensors(2, 333, 8, 2, seed=7)
    o, lse = forward(q, k, v, W, ns)
    grads = backward(q, k, v, o, lse, do, W, ns)
    x = [t.double() for t in (q, k, v)]
    f = lambda a, b, c: float((plain.window(a, b, c, W, ns, SCALE)["o"][0] * do.double()).sum())  # noqa: E731
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    want = plain.window(q, k, v, W, ns, SCALE, do)
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(x[i].shape, generator=g, device=DEV, dtype=torch.float64)
        e = 1e-4
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + e * d, x[i] - e * d
        num = (f(*hi) - f(*lo)) / (2 * e)
        got = float((grads[i].double() * d).sum())
        # roundings of single entries are independent of d: six standard deviations of their sum
        tol = 6 * float((want[name][1] * d).norm()) + 1e-5 * abs(num)
        assert abs(got - num) <= tol, (name, got, num, tol)


def test_equals_dense_warmup():
    """A window of the whole sequence is the dense attention the library already has."""
    q, k, v, _ = tensors(1, 1024, 8, 2, seed=8)
    o, lse = forward(q, k, v, 1024, 0)
    o2, lse2 = msa.msa_warmup_forward(q, k, v, SCALE)
    want = plain.window(q, k, v, 1024, 0, SCALE)
    assert (o.double() - o2.double()).abs().le(2 * want["o"][1]).all()
    assert (lse - lse2).abs().max() <= 2 * plain.F


def test_same_bits_every_time():
    q, k, v, do = tensors(2, 3000, 16, 2, seed=9)
    first = None
    for _ in range(3):
        o, lse = forward(q, k, v, 300, 140)
        out = (o, lse) + backward(q, k, v, o, lse, do, 300, 140)
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_batch_rows_are_alone():
    """A sequence's results do not depend on its neighbours in the batch (tiles end inside it)."""
    q, k, v, do = tensors(3, 201, 8, 2, seed=10)
    o, lse = forward(q, k, v, 64, 4)
    grads = backward(q, k, v, o, lse, do, 64, 4)
    o1, lse1 = forward(q[1:2].clone(), k[1:2].clone(), v[1:2].clone(), 64, 4)
    g1 = backward(q[1:2].clone(), k[1:2].clone(), v[1:2].clone(), o1, lse1, do[1:2].clone(), 64, 4)
    assert torch.equal(o[1:2], o1) and torch.equal(lse[1:2], lse1)
    assert all(torch.equal(a[1:2], b) for a, b in zip(grads, g1))


def test_func_and_graph():
    """The autograd function: strided inputs, gradients of the entry points, and a captured training step
    that follows new inputs, next to a second graph on the same stream."""
    W, ns = 90, 5
    q, k, v, do = tensors(2, 400, 8, 2, seed=11)
    packed = torch.cat([q, k, v], 2).requires_grad_()
    o = msa.msa_window_func(*packed.split((8, 2, 2), 2), W, ns, SCALE)
    o.backward(do)
    ro, rlse = forward(q, k, v, W, ns)
    want = torch.cat(backward(q, k, v, ro, rlse, do, W, ns), 2)
    assert torch.equal(o, ro) and torch.equal(packed.grad, want)

    def make(seed):
        x = [t.clone().requires_grad_() for t in tensors(2, 400, 8, 2, seed=seed)[:3]]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.autograd.grad(msa.msa_window_func(*x, W, ns, SCALE), x, do)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = msa.msa_window_func(*x, W, ns, SCALE)
            g = torch.autograd.grad(y, x, do)
        return x, graph, y, g

    a, b = make(20), make(21)
    for x, graph, y, g in (a, b):
        with torch.no_grad():
            for t, n in zip(x, tensors(2, 400, 8, 2, seed=22)):
                t.copy_(n)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(sa):
        a[1].replay()
    with torch.cuda.stream(sb):
        b[1].replay()
    torch.cuda.synchronize()
    q2, k2, v2 = tensors(2, 400, 8, 2, seed=22)[:3]
    o2, l2 = forward(q2, k2, v2, W, ns)
    g2 = backward(q2, k2, v2, o2, l2, do, W, ns)
    for _, _, y, g in (a, b):
        assert torch.equal(y, o2)
        assert all(torch.equal(s, t) for s, t in zip(g, g2))


def test_two_streams_at_once():
    q, k, v, do = tensors(1, 2048, 16, 2, seed=12)
    o, lse = forward(q, k, v, 256, 4)
    want = (o, lse) + backward(q, k, v, o, lse, do, 256, 4)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(3):
                o1, l1 = msa.msa_window_forward(q, k, v, 256, 4, SCALE)
                outs.append((o1, l1) + msa.msa_window_backward(q, k, v, o1, l1, do, 256, 4, SCALE))
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_long_sequence():
    """64K tokens: offsets past 2^31 bytes; rows spot-checked in 64 bits."""
    B, S, Hq, Hkv, W, ns = 1, 65536, 64, 8, 300, 4
    q, k, v, do = tensors(B, S, Hq, Hkv, seed=13)
    o, lse = forward(q, k, v, W, ns)
    dq = backward(q, k, v, o, lse, do, W, ns)[0]
    for t in (0, 3, 299, 300, 40000, S - 1):
        j = torch.arange(t + 1, device=DEV)
        j = j[(j > t - W) | (j < ns)]
        for h in (0, 13, 63):
            K, V = k[0, j, h // 8].double(), v[0, j, h // 8].double()
            s = K @ q[0, t, h].double() * SCALE
            p = (s - s.logsumexp(0)).exp()
            ref = p @ V
            eo = plain.HALF * ref.abs() + (plain.HALF + plain.F) * (p @ V.abs())
            assert ((o[0, t, h].double() - ref).abs() <= eo).all()
            assert abs(float(lse[0, h, t]) - float(s.logsumexp(0))) <= plain.F
            g = do[0, t, h].double()
            dp, dd = V @ g, (g * ref).sum()
            ds = SCALE * p * (dp - dd)
            es = plain.HALF * ds.abs() + SCALE * p * (plain.F * (dp.abs() + dd.abs()) + (g.abs() * eo).sum() * 1.01)
            rq, eq = ds @ K, es @ K.abs()
            assert ((dq[0, t, h].double() - rq).abs() <= eq + plain.HALF * (rq.abs() + eq)).all()


# ------------------------------------------------------------------------------------------ decode
# (B, capacity, Hq, Hkv, window, sinks, lengths)
DECODE = [
    (1, 1, 1, 1, 1, 0, [1]),
    (4, 200, 8, 2, 64, 4, [1, 64, 69, 200]),
    (3, 1000, 16, 1, 1000, 0, [1000, 999, 128]),
    (2, 3000, 4, 4, 300, 130, [3000, 431]),
    (5, 777, 32, 4, 1, 0, [777, 1, 2, 128, 129]),
    (2, 5000, 8, 8, 2 ** 31 - 1, 7, [4999, 3]),
    (8, 260, 16, 2, 128, 8, [260, 136, 137, 135, 128, 129, 8, 9]),
    (64, 300, 64, 8, 100, 4, [300 - 4 * i for i in range(64)]),  # one split: every pair resident
    (1, 70000, 16, 2, 60000, 16, [69999]),                       # many splits
]


@pytest.mark.parametrize("B,cap,Hq,Hkv,W,ns,lens", DECODE)
def test_decode(B, cap, Hq, Hkv, W, ns, lens):
    _, k, v, _ = tensors(B, cap, 1, Hkv, seed=cap)
    q = tensors(B, 1, Hq, Hkv, seed=cap + 1)[0][:, 0].contiguous()
    # everything the new token does not see is NaN or infinite
    for b, n in enumerate(lens):
        j = torch.arange(cap, device=DEV)
        out = ~((j < n) & ((j >= n - W) | (j < ns)))
        k[b, out] = float("nan")
        v[b, out] = float("inf")
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape = msa.make_window_shape(q, k, W, ns, SCALE)
    ws = msa.window_workspace(shape, msa.OP_WINDOW_DECODE, DEV)
    o, lse = msa.msa_window_decode(q, k, v, n, W, ns, SCALE, ws=ws)
    assert msa.msa_device_status(ws) == 0
    want = plain.window_decode(q, k, v, lens, W, ns, SCALE)
    plain.check("o", o, want["o"])
    plain.check("lse", lse, want["lse"])
    o2, lse2 = msa.msa_window_decode(q, k, v, n, W, ns, SCALE)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,Hkv,B,cap", [(8, 8, 40, 500), (16, 8, 40, 500), (64, 8, 20, 700), (16, 2, 2, 20000)])
def test_decode_rounds_once(Hq, Hkv, B, cap):
    """Groups of up to eight heads keep P to 2^-17: the error of o is that of rounding the 64-bit result, within 1
    percent (the second order of 2^-8; fp32 moves few values across a boundary).  P as one bf16 would add 40 percent."""
    _, k, v, _ = tensors(B, cap, 1, Hkv, seed=44)
    q = tensors(B, 1, Hq, Hkv, seed=45)[0][:, 0].contiguous()
    lens = [cap - i for i in range(B)]
    o, _ = msa.msa_window_decode(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV), cap, 0, SCALE)
    ref = plain.window_decode(q, k, v, lens, cap, 0, SCALE)["o"][0]
    err, floor = (float((x.double() - ref).norm() / ref.norm()) for x in (o, ref.to(torch.bfloat16)))
    assert err <= 1.01 * floor, (err, floor)


@pytest.mark.parametrize("cap,B", [(400, 3), (9000, 3)])
def test_decode_skips_bad_lengths(cap, B):
    """Lengths outside 1 .. S: flagged, their rows left as they were, the others right."""
    _, k, v, _ = tensors(B, cap, 1, 2, seed=30)
    q = tensors(B, 1, 8, 2, seed=31)[0][:, 0].contiguous()
    n = torch.tensor([0, cap, cap + 1], dtype=torch.int32, device=DEV)
    shape = msa.make_window_shape(q, k, cap, 0, SCALE)
    ws = msa.window_workspace(shape, msa.OP_WINDOW_DECODE, DEV)
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, 8), 7.0, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = msa.load_library().msa_window_decode(ctypes.byref(shape), p(q), p(k), p(v), p(n), p(o), p(lse), p(ws),
                                              ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    assert msa.msa_device_status(ws) == 1
    assert (o[[0, 2]] == 7).all() and (lse[[0, 2]] == 7).all()
    want = plain.window_decode(q[1:2], k[1:2], v[1:2], [cap], cap, 0, SCALE)
    plain.check("o", o[1:2], want["o"])
    plain.check("lse", lse[1:2], want["lse"])


def test_decode_is_the_forwards_row():
    W, ns, S = 130, 4, 500
    q, k, v, _ = tensors(2, S, 16, 2, seed=32)
    o, lse = forward(q, k, v, W, ns)
    want = plain.window(q, k, v, W, ns, SCALE)
    for t in (0, 1, 129, 130, 133, 134, 135, 400, 499):
        n = torch.full((2,), t + 1, dtype=torch.int32, device=DEV)
        o1, lse1 = msa.msa_window_decode(q[:, t].contiguous(), k, v, n, W, ns, SCALE)
        assert ((o1 - o[:, t]).double().abs() <= 2 * want["o"][1][:, t]).all()
        assert (lse1 - lse[:, :, t]).abs().max() <= 2 * plain.F


def test_decode_graph_follows_lengths():
    """One captured step replayed while the lengths grow."""
    _, k, v, _ = tensors(2, 2000, 1, 2, seed=33)
    q = tensors(2, 1, 8, 2, seed=34)[0][:, 0].contiguous()
    n = torch.tensor([100, 1900], dtype=torch.int32, device=DEV)
    msa.msa_window_decode(q, k, v, n, 512, 4, SCALE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = msa.msa_window_decode(q, k, v, n, 512, 4, SCALE)
    for lens in ([100, 1900], [101, 1901], [600, 2000], [1, 5]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want = plain.window_decode(q, k, v, lens, 512, 4, SCALE)
        plain.check("o", o, want["o"])
        plain.check("lse", lse, want["lse"])
