"""Norm and rotation of the heads against a plain 64-bit implementation, their gradients, the form that
writes into caches, and the operators run together as a model runs them."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rnd(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)


def weight(seed):
    return (1 + 0.2 * rnd(128, seed=seed, dtype=torch.float32)).contiguous()


def make(B, N, heads, seed=0):
    """A packed projection with tokens of different size, its slices, and gradients of the outputs."""
    x = rnd(B, N, sum(heads), 128, seed=seed)
    x = (x.float() * torch.exp(rnd(B, N, 1, 1, seed=seed + 1, dtype=torch.float32))).to(torch.bfloat16)
    dy = [rnd(B, N, h, 128, seed=seed + 2 + i) for i, h in enumerate(heads)]
    return x, x.split(heads, 2), dy


# (B, N, heads, rotary, interleaved, first position)
CASES = [
    (1, 1, [1], 128, False, 0),
    (1, 1, [64, 8, 8, 8, 1], 64, False, 1000000),
    (2, 3, [4, 2, 2, 2, 1], 128, True, 5),
    (1, 77, [8, 2, 2, 2, 1], 16, False, 0),
    (3, 33, [5, 3], 80, False, 123456789),
    (1, 129, [16, 1], 48, True, 2 ** 31 - 200),
    (2, 100, [2, 2], 0, False, 0),
    (1, 500, [3, 1, 1], 112, True, -400),       # positions before zero
    (1, 2100, [64, 8, 8, 8, 1], 128, False, 0),  # more tokens than resident warps
    (5, 1, [1, 1, 1, 1, 1, 1, 1, 1], 32, False, 9),
]


@pytest.mark.parametrize("B,N,heads,rot,inter,first", CASES)
def test_forward_and_backward(B, N, heads, rot, inter, first):
    x, xs, dy = make(B, N, heads, seed=N)
    f = freqs(rot) if rot else None
    pos = (first + torch.arange(N, device=DEV) + 3 * torch.arange(B, device=DEV)[:, None]).to(torch.int32)
    # norm and rotation, norm only, rotation only, neither
    ws = [weight(i) if i % 4 in (0, 1) else None for i in range(len(heads))]
    rotate = [bool(rot) and i % 4 in (0, 2) for i in range(len(heads))]
    kw = dict(positions=pos, eps=1e-5, rotate=rotate, interleaved=inter)
    ys = msa.msa_norm_rope_forward(xs, ws, f, **kw)
    dx = torch.full_like(x, float("nan"))
    dxs, dws = msa.msa_norm_rope_backward(xs, ws, dy, f, dxs=dx.split(heads, 2), **kw)
    fresh, dws2 = msa.msa_norm_rope_backward(xs, ws, dy, f, **kw)
    assert torch.equal(torch.cat(fresh, 2), dx)
    for i in range(len(heads)):
        want = plain.norm_rope(xs[i], ws[i], pos, f if rotate[i] else None, inter, 1e-5, dy[i])
        assert ys[i].is_contiguous()
        plain.check(f"y{i}", ys[i], want["y"])
        plain.check(f"dx{i}", dxs[i], want["dx"])
        assert (dws[i] is None) == (ws[i] is None)
        if ws[i] is not None:
            plain.check(f"dw{i}", dws[i], want["dw"])
            assert torch.equal(dws[i], dws2[i])  # the same bits every time
        elif not rotate[i]:
            assert torch.equal(ys[i], xs[i]) and torch.equal(dxs[i], dy[i])


def test_default_positions_and_strides():
    """No positions: 0 .. N - 1; inputs with strides of their own, one batch row, dense results."""
    big = rnd(2, 50, 12, 128, seed=3)
    x = big[:, ::2, 3:7]
    f, w = freqs(128), weight(1)
    y, = msa.msa_norm_rope_forward([x], [w], f)
    pos = torch.arange(25, device=DEV).expand(2, 25)
    plain.check("y", y, plain.norm_rope(x, w, pos, f, False, 1e-6)["y"])
    y1, = msa.msa_norm_rope_forward([x[1:]], [w], f)
    assert torch.equal(y1, y[1:])
    yt, = msa.msa_norm_rope_forward([big.transpose(0, 1)[:, :, :1]], [w], f)  # tokens outermost in memory
    pos = torch.arange(2, device=DEV).expand(50, 2)
    plain.check("y", yt, plain.norm_rope(big.transpose(0, 1)[:, :, :1], w, pos, f, False, 1e-6)["y"])


def test_extreme_rows():
    """Rows of zeros stay zeros with zero-size gradients; tiny and huge rows are normed alike."""
    x = rnd(1, 6, 2, 128, seed=4).float()
    x[0, 0] = 0
    x[0, 1] *= 1e-12
    x[0, 2] *= 1e12
    x = x.to(torch.bfloat16)
    w, f, dy = weight(2), freqs(64), rnd(1, 6, 2, 128, seed=5)
    pos = torch.arange(6, device=DEV).view(1, 6)
    for eps in (1e-6, 1e-30):
        y, = msa.msa_norm_rope_forward([x], [w], f, eps=eps)
        (dx,), (dw,) = msa.msa_norm_rope_backward([x], [w], [dy], f, eps=eps)
        want = plain.norm_rope(x, w, pos, f, False, eps, dy)
        plain.check("y", y, want["y"])
        plain.check("dx", dx, want["dx"])
        assert (y[0, 0] == 0).all()


def test_differences():
    """Directional derivatives of sum(y * dy) in 64 bits against the gradients of x and w."""
    x, (xq,), (dy,) = make(2, 40, [6], seed=6)
    f, w = freqs(96), weight(3)
    pos = torch.arange(7, 47, device=DEV).expand(2, 40).to(torch.int32).contiguous()
    (dx,), (dw,) = msa.msa_norm_rope_backward([xq], [w], [dy], f, positions=pos)
    want = plain.norm_rope(xq, w, pos, f, False, 1e-6, dy)
    loss = lambda a, b: float((plain.norm_rope(a, b, pos, f, False, 1e-6)["y"][0] * dy.double()).sum())  # noqa: E731
    d = rnd(*xq.shape, seed=7, dtype=torch.float64)
    e = 1e-5 * float(xq.double().square().mean().sqrt())
    num = (loss(xq.double() + e * d, w) - loss(xq.double() - e * d, w)) / (2 * e)
    got = float((dx.double() * d).sum())
    assert abs(got - num) <= 6 * float((want["dx"][1] * d).norm()) + 1e-4 * abs(num) + 1e-3
    d = rnd(128, seed=8, dtype=torch.float64)
    num = (loss(xq, w.double() + 1e-5 * d) - loss(xq, w.double() - 1e-5 * d)) / 2e-5
    got = float((dw.double() * d).sum())
    assert abs(got - num) <= float((want["dw"][1] * d.abs()).sum()) + 1e-5 * abs(num) + 1e-4


def test_in_place_rows():
    """dxs may be the dys themselves: a row is read whole before it is written."""
    x, xs, dy = make(2, 60, [4, 2], seed=9)
    f, ws = freqs(128), [weight(4), weight(5)]
    want, wdw = msa.msa_norm_rope_backward(xs, ws, dy, f)
    got, gdw = msa.msa_norm_rope_backward(xs, ws, dy, f, dxs=dy)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(wdw, gdw))


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
def test_funcs(wdtype):
    """Both autograd functions against the entry points; weights of another dtype; an unused output."""
    heads = [8, 2, 2, 2, 1]
    x, xs, dy = make(2, 90, heads, seed=10)
    f = freqs(64)
    ws = [weight(i).to(wdtype).requires_grad_() if i != 2 else None for i in range(5)]
    rotate = [True, True, False, True, True]
    xp = x.clone().requires_grad_()
    ys = msa.msa_norm_rope_packed_func(xp, heads, ws, f, rotate=rotate)
    torch.autograd.backward(ys[:4], dy[:4])
    w32 = [None if w is None else w.detach().float() for w in ws]
    want_y = msa.msa_norm_rope_forward(xs, w32, f, rotate=rotate)
    zero = dy[:4] + [torch.zeros_like(dy[4])]
    dxs, dws = msa.msa_norm_rope_backward(xs, w32, zero, f, rotate=rotate)
    assert all(torch.equal(a, b) for a, b in zip(ys, want_y))
    assert torch.equal(xp.grad, torch.cat(dxs, 2))
    for w, d in zip(ws, dws):
        assert w is None or (w.grad.dtype == wdtype and torch.equal(w.grad, d.to(wdtype)))
        if w is not None:
            w.grad = None
    sep = [t.clone().requires_grad_() for t in xs]
    ys = msa.msa_norm_rope_func(sep, ws, f, rotate=rotate)
    torch.autograd.backward(ys, zero)
    assert all(torch.equal(t.grad, d) for t, d in zip(sep, dxs))


# ------------------------------------------------------------------------------------------ append
def caches(B, cap, Hkv, seed=0):
    return [rnd(B, cap, Hkv, 128, seed=seed), rnd(B, cap, Hkv, 128, seed=seed + 1), rnd(B, cap, 128, seed=seed + 2)]


@pytest.mark.parametrize("B,N,cap,lens", [(1, 1, 128, [1]), (4, 1, 256, [1, 256, 17, 128]),
                                          (3, 5, 200, [5, 200, 131]), (130, 1, 128, [1 + i % 128 for i in range(130)]),
                                          (2, 40, 40, [40, 40])])
def test_append(B, N, cap, lens):
    heads = [8, 2, 2, 2, 1]
    x, xs, _ = make(B, N, heads, seed=11)
    f = freqs(128)
    ws = [weight(1), weight(2), None, weight(3), weight(4)]
    rotate = [True, True, False, True, True]
    kc, vc, pc = caches(B, cap, 2, seed=12)
    before = [t.clone() for t in (kc, vc, pc)]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st = torch.empty(256, dtype=torch.uint8, device=DEV)
    out = msa.msa_norm_rope_append(xs, ws, f, n, [None, kc, vc, None, pc], rotate=rotate, ws=st)
    assert msa.msa_device_status(st) == 0
    assert out[1] is kc and out[2] is vc and out[4] is pc
    pos = n.long()[:, None] - N + torch.arange(N, device=DEV)
    at = torch.arange(B, device=DEV)[:, None], pos
    rows = [out[0], kc[at], vc[at], out[3], pc[at].unsqueeze(2)]
    for i in range(5):
        want = plain.norm_rope(xs[i], ws[i], pos, f if rotate[i] else None, False, 1e-6)
        plain.check(f"part {i}", rows[i], want["y"])
    for c, old in zip((kc, vc, pc), before):  # every other row as it was
        c[at] = old[at]
        assert torch.equal(c, old)


def test_append_skips_bad_lengths():
    heads = [4, 2]
    x, xs, _ = make(4, 3, heads, seed=13)
    f, ws = freqs(64), [weight(1), weight(2)]
    kc = rnd(4, 64, 2, 128, seed=14)
    old = kc.clone()
    n = torch.tensor([2, 64, 65, -5], dtype=torch.int32, device=DEV)  # two tokens, too long, negative
    st = torch.empty(256, dtype=torch.uint8, device=DEV)
    out = msa.msa_norm_rope_append(xs, ws, f, n, [None, kc], ws=st)
    assert msa.msa_device_status(st) == 1
    assert torch.equal(kc[[0, 2, 3]], old[[0, 2, 3]]) and torch.equal(kc[1, :61], old[1, :61])
    pos = torch.arange(61, 64, device=DEV).view(1, 3)
    plain.check("k", kc[1:2, 61:], plain.norm_rope(xs[1][1:2], ws[1], pos, f, False, 1e-6)["y"])
    plain.check("q", out[0][1:2], plain.norm_rope(xs[0][1:2], ws[0], pos, f, False, 1e-6)["y"])


def test_append_refuses_one_cache_twice():
    x, xs, _ = make(1, 1, [2, 2], seed=60)
    kc = rnd(1, 64, 2, 128, seed=61)
    old = kc.clone()
    n = torch.ones(1, dtype=torch.int32, device=DEV)
    with pytest.raises(msa.MSAError, match="same output"):
        msa.msa_norm_rope_append(xs, None, None, n, [kc, kc])
    assert torch.equal(kc, old)


def test_backward_launches():
    """The join of the weights' gradients runs only where there is one; without it dx is dy turned back."""
    x, xs, dys = make(2, 9, [4, 2], seed=62)
    lib, f = msa.load_library(), freqs(64)
    count = []
    for w in ([None, None], [weight(1), None]):
        before = lib.msa_launch_count()
        dxs, dws = msa.msa_norm_rope_backward(xs, w, dys, f)
        count.append(lib.msa_launch_count() - before)
        assert [g is None for g in dws] == [v is None for v in w]
    assert count == [1, 2]


def test_append_graph_follows_lengths():
    """One captured append and window step replayed while the sequences grow: each replay writes the
    lengths' rows and no others, and attends to them."""
    B, cap, W, ns, scale = 3, 400, 60, 4, 128 ** -0.5
    f, ws, rotate = freqs(128), layer_params(70), [True, True, False, True, True]
    kc, vc, pc = caches(B, cap, 2, seed=63)
    x = rnd(B, sum(HEADS), 128, seed=64)
    n = torch.tensor([5, 100, 300], dtype=torch.int32, device=DEV)

    def step():
        q, _, _, _, _ = msa.msa_norm_rope_append(list(x.split(HEADS, 1)), ws, f, n, [None, kc, vc, None, pc], rotate=rotate)
        return (q,) + msa.msa_window_decode(q, kc, vc, n, W, ns, scale)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, lse = step()
    for i, lens in enumerate(([6, 101, 301], [7, 102, 302], [400, 1, 399])):
        x.copy_(rnd(B, sum(HEADS), 128, seed=65 + i))
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        before = [t.clone() for t in (kc, vc, pc)]
        graph.replay()
        torch.cuda.synchronize()
        pos = n.long()[:, None] - 1
        xs = [t.unsqueeze(1) for t in x.split(HEADS, 1)]
        at = (torch.arange(B, device=DEV), pos[:, 0])
        for j, row in ((0, q), (1, kc[at]), (2, vc[at]), (4, pc[at].unsqueeze(1))):
            want = plain.norm_rope(xs[j], ws[j], pos, f if rotate[j] else None, False, 1e-6)["y"]
            plain.check(f"part {j}", row.unsqueeze(1), want)
        want = plain.window_decode(q, kc, vc, lens, W, ns, scale)
        plain.check("o", o, want["o"])
        plain.check("lse", lse, want["lse"])
        for c, old in zip((kc, vc, pc), before):
            now = c.clone()
            now[at] = old[at]
            assert torch.equal(now, old)


def test_append_and_decode_on_two_streams():
    """Two requests' steps at once, each with caches of its own: the same bits as one after the other."""
    B, cap, W, ns, scale = 4, 2000, 700, 4, 128 ** -0.5
    f, ws, rotate = freqs(128), layer_params(80), [True, True, False, True, True]
    n = torch.tensor([2000, 900, 1, 1300], dtype=torch.int32, device=DEV)
    xs = [rnd(B, sum(HEADS), 128, seed=81 + i) for i in range(2)]

    def step(i, kv):
        q, _, _, _, _ = msa.msa_norm_rope_append(list(xs[i].split(HEADS, 1)), ws, f, n, [None, kv[0], kv[1], None, kv[2]],
                                                 rotate=rotate)
        return (q,) + msa.msa_window_decode(q, kv[0], kv[1], n, W, ns, scale)

    want = []
    for i in range(2):
        kv = caches(B, cap, 2, seed=90 + 3 * i)
        want.append(step(i, kv) + tuple(kv))
    kvs = [caches(B, cap, 2, seed=90 + 3 * i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(i, kvs[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want[i], got[i] + tuple(kvs[i])))


def test_long_caches():
    """Caches of more than 2^31 elements: the last rows of the last sequence are written and read."""
    B, cap, H, W, ns, scale = 3, 1 << 20, 8, 500, 4, 128 ** -0.5
    kc, vc = (torch.zeros(B, cap, H, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert kc.numel() > 2 ** 31
    lens = [cap, 7, cap - 1]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for b, m in enumerate(lens):
        for j, c in enumerate((kc, vc)):
            c[b, max(0, m - 600):m - 1] = rnd(m - 1 - max(0, m - 600), H, 128, seed=100 + 2 * b + j)
            c[b, :4] = rnd(4, H, 128, seed=110 + 2 * b + j)
    x = rnd(B, 3 * H, 128, seed=120)
    f, ws, rotate = freqs(128), [weight(1), weight(2), None], [True, True, False]
    q, _, _ = msa.msa_norm_rope_append(list(x.split(H, 1)), ws, f, n, [None, kc, vc], rotate=rotate)
    pos = n.long()[:, None] - 1
    at = (torch.arange(B, device=DEV), pos[:, 0])
    xs = [t.unsqueeze(1) for t in x.split(H, 1)]
    for j, row in enumerate((q, kc[at], vc[at])):
        want = plain.norm_rope(xs[j], ws[j], pos, f if rotate[j] else None, False, 1e-6)["y"]
        plain.check(f"part {j}", row.unsqueeze(1), want)
    assert not kc[1, 7:].any() and not kc[2, cap - 1].any() and not vc[0, 4:cap - 600].any()
    o, lse = msa.msa_window_decode(q, kc, vc, n, W, ns, scale)
    want = plain.window_decode(q, kc, vc, lens, W, ns, scale)
    plain.check("o", o, want["o"])
    plain.check("lse", lse, want["lse"])


# ------------------------------------------------------------------------------------------ together
HEADS = [16, 2, 2, 2, 1]  # q, k, v, qp, kp


def layer_params(seed):
    return [weight(seed), weight(seed + 1), None, weight(seed + 2), weight(seed + 3)]


def test_training_step_of_a_local_and_a_sparse_layer():
    """Projection -> norm and rotation -> window attention, and the same before sparse attention; the
    gradients equal the chain of the entry points, and a captured step replays them."""
    S, W, ns, top_k, scale = 512, 100, 4, 2, 128 ** -0.5
    f, ws = freqs(64), layer_params(40)
    rotate = [True, True, False, True, True]
    x = rnd(1, S, sum(HEADS), 128, seed=15).requires_grad_()
    do = rnd(1, S, 16, 128, seed=16)

    def step(sparse):
        q, k, v, qp, kp = msa.msa_norm_rope_packed_func(x, HEADS, ws, f, rotate=rotate)
        if sparse:
            o, kl = msa.msa_func(qp, kp, q, k, v, top_k, scale)
            return torch.autograd.grad([o, kl], [x], [do, torch.ones_like(kl)])[0], o.detach()
        o = msa.msa_window_func(q, k, v, W, ns, scale)
        # (detached: an eager graph of x kept alive would be synchronised with inside the capture)
        return torch.autograd.grad(o, [x], do)[0], o.detach()

    dx, o = step(False)
    xs = x.detach().split(HEADS, 2)
    q, k, v, qp, kp = msa.msa_norm_rope_forward(xs, ws, f, rotate=rotate)
    plain.check("o", o, plain.window(q, k, v, W, ns, scale)["o"])
    o1, lse1 = msa.msa_window_forward(q, k, v, W, ns, scale)
    dq, dk, dv = msa.msa_window_backward(q, k, v, o1, lse1, do, W, ns, scale)
    zeros = [torch.zeros_like(t) for t in (qp, kp)]
    dxs, _ = msa.msa_norm_rope_backward(xs, ws, [dq, dk, dv] + zeros, f, rotate=rotate)
    assert torch.equal(dx, torch.cat(dxs, 2))

    dxs_, os_ = step(True)
    o2, _, idx = msa.msa_forward(q, k, v, qp, kp, top_k, scale)
    assert torch.equal(os_, o2) and torch.isfinite(dxs_.float()).all()
    assert dxs_[..., -3:, :].float().abs().sum() > 0  # the KL term reaches the proxy heads' slices

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, go = step(False)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gx, dx) and torch.equal(go, o)


def test_decode_follows_prefill():
    """Prefill a prompt (one append of all its tokens), then decode token by token: append, then the
    window step and the sparse step over the same caches; both follow the whole-sequence forward."""
    B, S, P, W, ns, top_k, scale = 2, 384, 300, 60, 4, 2, 128 ** -0.5
    f, ws = freqs(128), layer_params(50)
    rotate = [True, True, False, True, True]
    x = rnd(B, S, sum(HEADS), 128, seed=17)
    q, k, v, qp, kp = msa.msa_norm_rope_forward(x.split(HEADS, 2), ws, f, rotate=rotate)
    wo = plain.window(q, k, v, W, ns, scale)
    so, slse, sidx = msa.msa_forward(q, k, v, qp, kp, top_k, scale)
    kc, vc = (torch.full((B, S, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc = torch.zeros((B, S, 128), dtype=torch.bfloat16, device=DEV)
    n = torch.full((B,), P, dtype=torch.int32, device=DEV)
    msa.msa_norm_rope_append(x[:, :P].split(HEADS, 2), ws, f, n, [None, kc, vc, None, pc], rotate=rotate)
    assert torch.equal(kc[:, :P], k[:, :P]) and torch.equal(vc[:, :P], v[:, :P]) and torch.equal(pc[:, :P], kp[:, :P, 0])
    for t in range(P, P + 5):
        n += 1
        q1, _, _, qp1, _ = msa.msa_norm_rope_append([s[:, 0] for s in x[:, t:t + 1].split(HEADS, 2)], ws, f, n,
                                                    [None, kc, vc, None, pc], rotate=rotate)
        assert torch.equal(q1, q[:, t]) and torch.equal(kc[:, t], k[:, t]) and torch.equal(pc[:, t], kp[:, t, 0])
        o, lse = msa.msa_window_decode(q1, kc, vc, n, W, ns, scale)
        plain.check("window o", o, tuple(z[:, t] for z in wo["o"]))
        plain.check("window lse", lse, tuple(z[:, :, t] for z in wo["lse"]))
    # the sparse step reads whole 128-key blocks of caches whose rest is finite
    kc, vc = kc.nan_to_num(0.0), vc.nan_to_num(0.0)
    o, lse, idx = msa.msa_decode(q1, qp1, kc, vc, pc.unsqueeze(2), n, top_k, scale)
    t = int(n[0]) - 1
    assert torch.equal(idx, sidx[:, :, t])
    assert (o - so[:, t]).float().abs().max() <= 0.02
