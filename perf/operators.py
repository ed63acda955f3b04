"""Work of the norm-and-rotation and sliding-window operators: their cases, inputs, plain forms and exact values.

norm_rope   per-head RMS norm of queries, keys and proxy heads with the position rotation, forward and backward over
            one packed projection, and the serving form that also writes the new rows into the caches.
window      causal GQA attention over a sliding window and a few first tokens that stay visible, forward, training
            (forward and backward) and one decode step over caches.

Head dim 128, bf16 tensors, fp32 norm weights and statistics.
"""
import math

import torch

own = False
D = 128


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding at small scale: latency of the norm, rotation and cache write of one token
        dict(name="append_b1", op="append", B=1, N=1, Hq=8, Hkv=2, Hp=2, cap=1024, rot=128, inter=False),
        # the decode batch of the library's decode workload, half of each head rotated
        dict(name="append_b128", op="append", B=128, N=1, Hq=64, Hkv=8, Hp=8, cap=512, rot=64, inter=False),
        # a small training step with a ragged length, interleaved pairs
        dict(name="rope_train_s999", op="rope", B=3, S=999, Hq=8, Hkv=2, Hp=2, rot=64, inter=True),
        # the heads of the 64K training step, one packed projection
        dict(name="rope_train_s64k", op="rope", B=1, S=65536, Hq=64, Hkv=8, Hp=8, rot=128, inter=False),
        # prefill of one short request of an odd length
        dict(name="win_fwd_s999", op="fwd", B=1, S=999, Hq=8, Hkv=2, W=128, sinks=4),
        # prefill of one long prompt in a layer with a wide window
        dict(name="win_fwd_s32k", op="fwd", B=1, S=32768, Hq=32, Hkv=8, W=2048, sinks=4),
        # the smallest training step: 1K tokens, few heads
        dict(name="win_train_s1k", op="train", B=1, S=1024, Hq=8, Hkv=2, W=256, sinks=16),
        # an ordinary training step
        dict(name="win_train_s8k", op="train", B=2, S=8192, Hq=32, Hkv=8, W=1024, sinks=4),
        # the long training step: 64K tokens, 64 query heads
        dict(name="win_train_s64k", op="train", B=1, S=65536, Hq=64, Hkv=8, W=512, sinks=4),
        # a few short requests, some shorter than the window
        dict(name="win_decode_b4", op="decode", B=4, Hq=8, Hkv=2, cap=1024, W=128, sinks=4),
        # the decode batch with a window of 1024
        dict(name="win_decode_b128", op="decode", B=128, Hq=64, Hkv=8, cap=4096, W=1024, sinks=4),
        # one long request with a wide window: the keys have to be split over the GPU
        dict(name="win_decode_b1", op="decode", B=1, Hq=64, Hkv=8, cap=65536, W=32768, sinks=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "fwd", "train", "train", "decode", "decode"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8, 16] if Hkv <= 4 else [1, 2, 4, 8])
    c = dict(op=op, Hq=Hq, Hkv=Hkv)
    if op in ("append", "rope"):
        c |= dict(Hp=rng.choice([1, Hkv]), rot=16 * rng.randint(1, 8), inter=rng.random() < 0.4)
    if op == "append":
        N = rng.choice([1, 1, 1, 2, 5])
        c |= dict(B=_log(rng, 1, 128), N=N, cap=rng.choice([128, 256, 512]))
    elif op == "rope":
        B = rng.choice([1, 2, 3])
        c |= dict(B=B, S=_log(rng, 1, 65536 // B))
    elif op == "decode":
        B, cap = _log(rng, 1, 128), _log(rng, 128, 4096)
        if B <= 4:
            cap *= 8
        c |= dict(B=B, cap=cap, W=_log(rng, 1, cap), sinks=rng.choice([0, 1, 4, 16, 130]))
    else:
        # a training step of one visible key a query has gradients of zero, where only rounding would be compared
        least = 2 if op == "train" else 1
        B, W = rng.choice([1, 1, 2, 3]), _log(rng, least, 4096)
        most = (16 * 2 ** 30) // (B * Hq * (2 * W + 512) * 4)  # keeps the plain form's scores within the largest case's
        c |= dict(B=B, S=_log(rng, least, max(least, min(32768, most))), W=W, sinks=rng.choice([0, 1, 4, 16, 130]))
    return c


def _visible(n, W, sinks):
    """Visible (query, key) pairs of the queries 0 .. n - 1 of one sequence and head."""
    full = n * (n + 1) // 2
    far = max(0, n - W)  # keys 0 .. t - W fall out of the window of t >= W
    lost = far * (far + 1) // 2
    k = min(sinks, far)  # sink j < k stays visible to its n - W - j far queries
    return full - lost + k * far - k * (k - 1) // 2


def _heads(c):
    return [c["Hq"], c["Hkv"], c["Hkv"], c["Hp"], 1]


def _lens(c):
    """Lengths of the sequences of a batch: ragged, the full capacity and (from four on) a single token among them."""
    B, cap, lo = c["B"], c["cap"], c.get("N", 1)
    lens = [max(lo, cap - (i * 7919) % max(1, cap // 2)) for i in range(B)]
    if B >= 4:
        lens[1] = lo
        lens[2] = min(cap, max(lo, cap // 16 + 1))
    return lens


def work(c):
    if c["op"] in ("append", "rope"):
        rows = c["B"] * (c["N"] if c["op"] == "append" else c["S"]) * sum(_heads(c))
        if c["op"] == "append":
            return {"bytes": rows * 2 * 256, "flops": rows * 8 * D}
        return {"bytes": rows * 5 * 256, "flops": rows * 24 * D}
    if c["op"] == "decode":
        seen = sum(min(n, c["W"] + min(c["sinks"], max(0, n - c["W"]))) for n in _lens(c))
        return {"bytes": seen * c["Hkv"] * 512 + c["B"] * c["Hq"] * 516, "flops": 4 * D * seen * c["Hq"]}
    pairs = c["B"] * c["Hq"] * _visible(c["S"], c["W"], c["sinks"])
    q, kv = c["B"] * c["S"] * c["Hq"], c["B"] * c["S"] * c["Hkv"]
    if c["op"] == "fwd":
        return {"bytes": q * 516 + kv * 512, "flops": 4 * D * pairs}
    # q, k, v, dout in; o, lse, dq, dk, dv out
    return {"bytes": q * (4 * 256 + 4) + kv * 4 * 256, "flops": 14 * D * pairs}


# ------------------------------------------------------------------------------------------ inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)

    s = {"case": c, "scale": D ** -0.5}
    if c["op"] in ("append", "rope"):
        heads = _heads(c)
        n = c["N"] if c["op"] == "append" else c["S"]
        x = randn(c["B"], n, sum(heads), D)
        # tokens of a residual stream differ in magnitude
        x *= torch.exp(0.5 * torch.randn((c["B"], n, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)
        s["x"], s["heads"] = x, heads
        # q, k, qp and kp are normed and rotated; v goes through as it is
        w = lambda: 1 + 0.1 * torch.randn(D, generator=g, device="cuda")  # noqa: E731
        s["weights"] = [w(), w(), None, w(), w()]
        s["rotate"] = [True, True, False, True, True]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
        if c["op"] == "rope":
            first = torch.randint(0, 1000000, (c["B"], 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(n, device="cuda")).to(torch.int32)
            s["dy"] = [randn(c["B"], n, h, D) for h in heads]
        else:
            s["seq_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
            s["caches"] = [None] + [randn(c["B"], c["cap"], h, D) for h in heads[1:3]] + [None, randn(c["B"], c["cap"], 1, D)]
        return s
    if c["op"] == "decode":
        s["q"] = randn(c["B"], c["Hq"], D)
        s["k"], s["v"] = (randn(c["B"], c["cap"], c["Hkv"], D) for _ in range(2))
        s["seq_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        return s
    s["q"], s["dout"] = randn(c["B"], c["S"], c["Hq"], D), randn(c["B"], c["S"], c["Hq"], D)
    s["k"], s["v"] = (randn(c["B"], c["S"], c["Hkv"], D) for _ in range(2))
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _rot_plain(u, cos, sin, rot, inter):
    """Rotates the first `rot` elements of u [..., H, D] by the angles of cos, sin [..., 1, rot / 2]."""
    a, b = (u[..., 0:rot:2], u[..., 1:rot:2]) if inter else (u[..., :rot // 2], u[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if inter else torch.cat([ya, yb], -1)
    return torch.cat([y, u[..., rot:]], -1)


def _norm_rope_plain(x, w, rotate, cos, sin, rot, inter, eps):
    x = x.float()
    u = x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w
    return (_rot_plain(u, cos, sin, rot, inter) if rotate else u).to(torch.bfloat16)


def _norm_rope_back_plain(x, w, dy, rotate, cos, sin, rot, inter, eps):
    x, dy = x.float(), dy.float()
    g = _rot_plain(dy, cos, -sin, rot, inter) if rotate else dy
    if w is None:
        return g.to(torch.bfloat16), None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * r
    h = g * w
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * n).sum((0, 1, 2))


def _angles(positions, inv_freq):
    a = positions.double().unsqueeze(-1) * inv_freq.double()  # far positions: 32 bits lose the angle
    return a.cos().float().unsqueeze(-2), a.sin().float().unsqueeze(-2)


def _window_keys(c, device):
    """Blocks of bs queries and the keys of each: (query positions [nb, bs], key positions [nb, L], visible [nb, bs, L])."""
    S, W, ns = c["S"], min(c["W"], c["S"]), min(c["sinks"], c["S"])
    bs = min(256, S)
    nb = -(-S // bs)
    t = torch.arange(nb * bs, device=device).view(nb, bs)
    j = t[:, :1] - (W - 1) + torch.arange(W - 1 + bs, device=device)
    near = (j[:, None] <= t[..., None]) & (t[..., None] - j[:, None] < W) & (j[:, None] >= 0)
    f = torch.arange(ns, device=device).expand(nb, ns)
    far = (t[..., None] - f[:, None] >= W) & (f[:, None] <= t[..., None])
    j = torch.cat([j, f], 1)
    return t.clamp(max=S - 1), j.clamp(0, S - 1), torch.cat([near, far], 2), bs, nb


def _window_scores_plain(q, k, c, scale):
    t, j, seen, bs, nb = _window_keys(c, q.device)
    B, G = c["B"], c["Hq"] // c["Hkv"]
    qb = q.float()[:, t].view(B, nb, bs, c["Hkv"], G, D)
    kb = k.float()[:, j]
    s = torch.einsum("bnthgd,bnjhd->bnhgtj", qb, kb).mul_(scale)
    return s.masked_fill_(~seen[None, :, None, None], -math.inf), qb, kb, t, j


def _unblock(x, c):
    """[B, nb, Hkv, G, bs, d] -> [B, S, Hq, d]"""
    return x.permute(0, 1, 4, 2, 3, 5).flatten(1, 2)[:, :c["S"]].flatten(2, 3)


def _window_plain(s, train):
    c, scale = s["case"], s["scale"]
    sc, qb, kb, t, j = _window_scores_plain(s["q"], s["k"], c, scale)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p.div_(l)
    vb = s["v"].float()[:, j]
    ob = torch.einsum("bnhgtj,bnjhd->bnhgtd", p, vb)
    o = _unblock(ob, c)
    lse = _unblock(m + l.log(), c).squeeze(-1).transpose(1, 2).contiguous()
    if not train:
        return o.to(torch.bfloat16).contiguous(), lse
    B, S, G = c["B"], c["S"], c["Hq"] // c["Hkv"]
    nb, bs = t.shape
    dob = s["dout"].float()[:, t].view(B, nb, bs, c["Hkv"], G, D)
    if nb * bs > S:  # the positions behind the last token stand for none
        dob = dob * (torch.arange(nb * bs, device=dob.device).view(1, nb, bs, 1, 1, 1) < S)
    dv = torch.zeros(s["v"].shape, dtype=torch.float32, device=o.device)
    dk = torch.zeros_like(dv)
    at = j.flatten()
    dv.index_add_(1, at, torch.einsum("bnhgtj,bnthgd->bnjhd", p, dob).flatten(1, 2))
    ds = torch.einsum("bnthgd,bnjhd->bnhgtj", dob, vb)
    ds.sub_((dob.permute(0, 1, 3, 4, 2, 5) * ob).sum(-1, keepdim=True)).mul_(p)
    dq = _unblock(torch.einsum("bnhgtj,bnjhd->bnhgtd", ds, kb), c) * scale
    dk.index_add_(1, at, torch.einsum("bnhgtj,bnthgd->bnjhd", ds, qb).flatten(1, 2))
    half = lambda x: x.to(torch.bfloat16).contiguous()  # noqa: E731
    return half(o), lse, half(dq), half(dk * scale), half(dv)


def _decode_plain(s):
    c = s["case"]
    B, G, n = c["B"], c["Hq"] // c["Hkv"], s["seq_len"].long().view(-1, 1)
    j = torch.arange(c["cap"], device=n.device)
    seen = (j < n) & ((j >= n - c["W"]) | (j < c["sinks"]))
    q = s["q"].float().view(B, c["Hkv"], G, D)
    sc = torch.einsum("bhgd,bjhd->bhgj", q, s["k"].float()) * s["scale"]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgj,bjhd->bhgd", p / l, s["v"].float())
    return o.reshape(B, c["Hq"], D).to(torch.bfloat16), (m + l.log()).reshape(B, c["Hq"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "decode":
        return _decode_plain(s)
    if c["op"] in ("fwd", "train"):
        return _window_plain(s, c["op"] == "train")
    eps, rot, inter = 1e-6, c["rot"], c["inter"]
    xs = s["x"].split(s["heads"], 2)
    if c["op"] == "rope":
        cos, sin = _angles(s["positions"], s["inv_freq"])
        ys = [_norm_rope_plain(x, w, r, cos, sin, rot, inter, eps) for x, w, r in zip(xs, s["weights"], s["rotate"])]
        back = [_norm_rope_back_plain(x, w, dy, r, cos, sin, rot, inter, eps)
                for x, w, dy, r in zip(xs, s["weights"], s["dy"], s["rotate"])]
        return ys, torch.cat([b[0] for b in back], 2), [b[1] for b in back if b[1] is not None]
    pos = s["seq_len"].long().view(-1, 1) - c["N"] + torch.arange(c["N"], device="cuda")
    cos, sin = _angles(pos, s["inv_freq"])
    ys = [_norm_rope_plain(x, w, r, cos, sin, rot, inter, eps) for x, w, r in zip(xs, s["weights"], s["rotate"])]
    b = torch.arange(c["B"], device="cuda").view(-1, 1)
    return [y if cache is None else cache.index_put_((b, pos), y) for y, cache in zip(ys, s["caches"])]


def run(s):
    if not own:
        return _run_plain(s)
    from block_sparse_attention_qp_gb300 import binding as msa
    c = s["case"]
    if c["op"] == "decode":
        return msa.msa_window_decode(s["q"], s["k"], s["v"], s["seq_len"], c["W"], c["sinks"], s["scale"])
    if c["op"] in ("fwd", "train"):
        o, lse = msa.msa_window_forward(s["q"], s["k"], s["v"], c["W"], c["sinks"], s["scale"])
        if c["op"] == "fwd":
            return o, lse
        return (o, lse) + msa.msa_window_backward(s["q"], s["k"], s["v"], o, lse, s["dout"], c["W"], c["sinks"], s["scale"])
    xs = s["x"].split(s["heads"], 2)
    if c["op"] == "append":
        return msa.msa_norm_rope_append(xs, s["weights"], s["inv_freq"], s["seq_len"], s["caches"], rotate=s["rotate"],
                                        interleaved=c["inter"])
    how = dict(positions=s["positions"], rotate=s["rotate"], interleaved=c["inter"])
    ys = msa.msa_norm_rope_forward(xs, s["weights"], s["inv_freq"], **how)
    dx = torch.empty_like(s["x"])
    _, dws = msa.msa_norm_rope_backward(xs, s["weights"], s["dy"], s["inv_freq"], dxs=dx.split(s["heads"], 2), **how)
    return list(ys), dx, [d for d in dws if d is not None]


# ------------------------------------------------------------------------------------------ exact values
def _exact_rope(s):
    """Rotation as a complex product, gradients from the derivative of x / rms(x), a token chunk at a time."""
    c = s["case"]
    rot, inter, eps = c["rot"], c["inter"], 1e-6
    f = s["inv_freq"].double()
    if c["op"] == "append":
        pos = s["seq_len"].long()[:, None] - c["N"] + torch.arange(c["N"], device="cuda")[None]
    else:
        pos = s["positions"].long()

    def turn(u, p, sign):
        z = u[..., :rot].unflatten(-1, (rot // 2, 2)) if inter else u[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous())
        ang = p.double()[..., None, None] * f
        z = torch.view_as_real(z * torch.polar(torch.ones_like(ang), sign * ang))
        z = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, u[..., rot:]], -1)

    ys, dxs, dws = [], [], []
    at = 0
    for i, h in enumerate(s["heads"]):
        x, w = s["x"][:, :, at:at + h], s["weights"][i]
        at += h
        y, dx = torch.empty(x.shape, dtype=torch.float64, device="cuda"), torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(D, dtype=torch.float64, device="cuda")
        for a in range(0, x.shape[1], 4096):
            xc, pc = x[:, a:a + 4096].double(), pos[:, a:a + 4096]
            rms = (xc.pow(2).sum(-1, keepdim=True) / D + eps).sqrt()
            u = xc if w is None else xc / rms * w.double()
            y[:, a:a + 4096] = turn(u, pc, 1) if s["rotate"][i] else u
            if c["op"] == "rope":
                gr = s["dy"][i][:, a:a + 4096].double()
                gr = turn(gr, pc, -1) if s["rotate"][i] else gr
                if w is not None:
                    dw += (gr * xc / rms).sum((0, 1, 2))
                    gr = gr * w.double()
                    gr = gr / rms - xc * (gr * xc).sum(-1, keepdim=True) / (D * rms ** 3)
                dx[:, a:a + 4096] = gr
        if c["op"] == "append" and s["caches"][i] is not None:
            full = s["caches"][i].double()
            for b in range(c["B"]):
                full[b, pos[b]] = y[b]
            y = full
        ys.append(y)
        dxs.append(dx)
        if w is not None:
            dws.append(dw)
    return ys if c["op"] == "append" else (ys, torch.cat(dxs, 2), dws)


def _exact_window(s, train):
    """A chunk of queries against every key it can reach, from the definition."""
    c, scale = s["case"], s["scale"]
    S, W, ns, G = c["S"], c["W"], c["sinks"], c["Hq"] // c["Hkv"]
    o, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty((c["B"], c["Hq"], S), dtype=torch.float64, device="cuda")
    dq = torch.empty_like(o)
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    step = 512
    for b in range(c["B"]):
        for a in range(0, S, step):
            t = torch.arange(a, min(S, a + step), device="cuda")
            lo = max(0, a - W + 1)
            j = torch.cat([torch.arange(min(ns, lo), device="cuda"), torch.arange(lo, int(t[-1]) + 1, device="cuda")])
            diff = t[:, None] - j
            seen = (diff >= 0) & ((diff < W) | (j < ns))
            kj, vj = s["k"][b, j].double(), s["v"][b, j].double()
            for h in range(c["Hkv"]):
                hs = slice(h * G, h * G + G)
                q = s["q"][b, t][:, hs].double().transpose(0, 1)
                sc = (q @ kj[:, h].T * scale).masked_fill(~seen, -math.inf)
                ls = sc.logsumexp(-1, keepdim=True)
                p = (sc - ls).exp()
                ob = p @ vj[:, h]
                o[b, a:a + step, hs] = ob.transpose(0, 1)
                lse[b, hs, a:a + step] = ls[..., 0]
                if train:
                    do = s["dout"][b, t][:, hs].double().transpose(0, 1)
                    dv[b, :, h].index_add_(0, j, torch.einsum("gtj,gtd->jd", p, do))
                    ds = p * (do @ vj[:, h].T - (do * ob).sum(-1, keepdim=True)) * scale
                    dq[b, a:a + step, hs] = (ds @ kj[:, h]).transpose(0, 1)
                    dk[b, :, h].index_add_(0, j, torch.einsum("gtj,gtd->jd", ds, q))
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _exact_decode(s):
    c = s["case"]
    G, lens = c["Hq"] // c["Hkv"], s["seq_len"].tolist()
    o, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty((c["B"], c["Hq"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo = max(0, n - c["W"])
        j = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, n, device="cuda")])
        kj, vj = s["k"][b, j].double().transpose(0, 1), s["v"][b, j].double().transpose(0, 1)
        sc = s["q"][b].double().view(c["Hkv"], G, D) @ kj.transpose(1, 2) * s["scale"]
        lse[b] = sc.logsumexp(-1).flatten()
        o[b] = (sc.softmax(-1) @ vj).reshape(c["Hq"], D)
    return o, lse


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "decode":
        return _exact_decode(s)
    if c["op"] in ("fwd", "train"):
        return _exact_window(s, c["op"] == "train")
    return _exact_rope(s)
