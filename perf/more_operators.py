"""Work of the 4-bit cache, packed-prompt and several-axes operators: their cases, inputs, plain forms and exact values.

axes     norm and rotation of queries, keys and proxy heads by positions of several axes (time, height, width): forward
         and backward over one packed projection, and the serving form that writes the new rows into the caches.
packed   causal GQA attention over sequences of different lengths that lie one behind the other, forward and training.
q4       caches in 4 bits: storing a prompt's rows, and decode steps that store the new token's rows and attend over
         the window and the first tokens (step) or over the key blocks that the proxy selects (sparse).

Head dim 128, bf16 tensors, fp32 norm weights and statistics.  A cache row in 4 bits is 128 codes of sign, two exponent
bits and one of mantissa, a scale for each 16 of them (sign, four exponent bits, three of mantissa) and a power of two
for the row; 128 rows of one head lie together as [128][64] bytes of codes, [128][8] scales, [128] exponents + 127.
"""
import math
import random

import torch

own = False
D = 128
BLOCK = 128
CHUNK = BLOCK * (D // 2 + D // 16 + 1)  # bytes of a block of 128 rows
E_MIN, E_MAX = -100, 90


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one image's tokens beside text in a small model, odd length, half of each head rotated
        dict(name="axes_train_s999", op="axes", B=2, S=999, Hq=8, Hkv=2, Hp=2, rot=64, inter=False, A=2),
        # a long video prompt, every element rotated by one of three axes
        dict(name="axes_train_s32k", op="axes", B=1, S=32768, Hq=32, Hkv=8, Hp=8, rot=128, inter=False, A=3),
        # the decode batch: the new tokens' positions are their own, not their cache rows
        dict(name="axes_append_b128", op="axes_append", B=128, Hq=64, Hkv=8, Hp=8, cap=512, rot=128, inter=False, A=3),
        # a handful of short requests prefilled in one call
        dict(name="packed_fwd_s700", op="packed", train=False, T=700, pad=3, top=150, mix=1, Hq=8, Hkv=2, W=0),
        # prefill of many requests, the longest of 4096 tokens
        dict(name="packed_fwd_s16k", op="packed", train=False, T=16384, pad=0, top=4096, mix=2, Hq=32, Hkv=8, W=0),
        # a small training step over packed documents in a layer with a window
        dict(name="packed_train_s2k", op="packed", train=True, T=2048, pad=5, top=900, mix=3, Hq=8, Hkv=2, W=256),
        # an ordinary training step over packed documents
        dict(name="packed_train_s16k", op="packed", train=True, T=16384, pad=37, top=4096, mix=4, Hq=32, Hkv=8, W=0),
        # one short request decoding at small scale: latency of storing a token and attending
        dict(name="q4_step_b1", op="step", B=1, Hq=8, Hkv=2, cap=1024, W=128, sinks=4),
        # the decode batch over whole caches
        dict(name="q4_step_b128", op="step", B=128, Hq=64, Hkv=8, cap=4096, W=4096, sinks=0),
        # one long request: the keys have to be split over the GPU
        dict(name="q4_long_b1", op="step", B=1, Hq=64, Hkv=8, cap=65536, W=65536, sinks=0),
        # sparse decode of a batch with 8K cached tokens
        dict(name="q4_sparse_b32", op="sparse", B=32, Hq=64, Hkv=8, Hp=8, cap=8192, top_k=16),
        # two prompts of 8K tokens stored
        dict(name="q4_store_s8k", op="store", B=2, N=8192, Hkv=8, cap=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "axes_append", "packed", "packed", "packed", "step", "step", "sparse", "store"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8, 16] if Hkv <= 2 else [1, 2, 4, 8] if Hkv == 4 else [1, 2, 4])
    c = dict(op=op, Hq=Hq, Hkv=Hkv)
    if op in ("axes", "axes_append"):
        c |= dict(Hp=rng.choice([1, Hkv]), rot=16 * rng.randint(1, 8), inter=rng.random() < 0.4, A=rng.choice([2, 3, 4]))
        if op == "axes_append":
            return c | dict(B=_log(rng, 1, 128), cap=rng.choice([128, 256, 512]))
        B = rng.choice([1, 2, 3])
        return c | dict(B=B, S=_log(rng, 1, 32768 // B))
    if op == "packed":
        train = rng.random() < 0.6
        least = 2 if train else 1  # a training step of one visible key a query has gradients of zero
        T = _log(rng, 8, 16384)
        top = _log(rng, least, min(T, 4096))
        W = 0 if rng.random() < 0.6 else _log(rng, least, 4096)
        return c | dict(train=train, T=T, pad=rng.choice([0, 1, 5]) if T > 8 else 0, top=top, mix=rng.randint(10, 10 ** 6), W=W)
    cap = 128 * _log(rng, 1, 64)
    if op == "step":
        B = _log(rng, 1, 64)
        if B <= 4:
            cap *= 8
        return c | dict(B=B, cap=cap, W=_log(rng, 1, cap), sinks=rng.choice([0, 1, 4, 16, 130]))
    if op == "sparse":
        c["Hp"] = rng.choice([1, Hkv]) if Hq <= 16 else Hkv
        return c | dict(B=_log(rng, 1, 32), cap=cap, top_k=rng.choice([1, 2, 4, 8, 16, 17, 32]))
    N = _log(rng, 1, cap)
    return dict(op=op, Hkv=Hkv, B=rng.choice([1, 2, 3]), N=N, cap=cap)


def _heads(c):
    return [c["Hq"], c["Hkv"], c["Hkv"], c["Hp"], 1]


def _axes(c):
    """The axis of each pair: one quarter of them the first axis's, the others shared by the rest."""
    n = c["rot"] // 2
    first = max(1, n // 4)
    return [0] * first + [1 + (i * (c["A"] - 1)) // (n - first) for i in range(n - first)]


def _lens(c):
    """Lengths of the sequences of a batch: ragged, the full capacity and (from four on) a single token among them."""
    B, cap = c["B"], c["cap"]
    lens = [max(1, cap - (i * 7919) % max(1, cap // 2)) for i in range(B)]
    if B >= 4:
        lens[1] = 1
        lens[2] = max(1, cap // 16 + 1)
    return lens


def _documents(c):
    """Lengths of packed sequences: spread over their logarithm up to `top`, the first of that length, T - pad together."""
    r, left, lens = random.Random(c["mix"]), c["T"] - c["pad"], []
    n = c["top"]
    while left > 0:
        n = min(n, left)
        lens.append(n)
        left -= n
        n = _log(r, 1, c["top"])
    return lens


def _window(c):
    return c["W"] if c["W"] else c["T"]


def _causal_pairs(n, W):
    far = max(0, n - W)
    return n * (n + 1) // 2 - far * (far + 1) // 2


def work(c):
    if c["op"] in ("axes", "axes_append"):
        rows = c["B"] * c.get("S", 1) * sum(_heads(c))
        if c["op"] == "axes_append":
            return {"bytes": rows * 2 * 256, "flops": rows * 8 * D}
        normed = rows // sum(_heads(c)) * (sum(_heads(c)) - c["Hkv"])  # v has no weight: its backward needs dy alone
        return {"bytes": rows * 4 * 256 + normed * 256, "flops": rows * 24 * D}
    if c["op"] == "packed":
        pairs = c["Hq"] * sum(_causal_pairs(n, _window(c)) for n in _documents(c))
        n = c["T"] - c["pad"]
        q, kv = n * c["Hq"], n * c["Hkv"]
        if not c["train"]:
            return {"bytes": q * 516 + kv * 512, "flops": 4 * D * pairs}
        return {"bytes": q * (4 * 256 + 4) + kv * 4 * 256, "flops": 14 * D * pairs}
    row = CHUNK // BLOCK
    if c["op"] == "store":  # bf16 in, 4 bits out, and read back as the bf16 values they stand for
        return {"bytes": c["B"] * c["N"] * c["Hkv"] * 2 * (256 + 2 * row + 256), "flops": c["B"] * c["N"] * c["Hkv"] * 2 * 4 * D}
    new = c["B"] * c["Hkv"] * 2 * (256 + row) + c["B"] * c["Hq"] * 516
    if c["op"] == "step":
        seen = sum(min(n, c["W"] + min(c["sinks"], max(0, n - c["W"]))) for n in _lens(c))
        return {"bytes": seen * c["Hkv"] * 2 * row + new, "flops": 4 * D * seen * c["Hq"]}
    lens = _lens(c)
    seen = sum(min(n, (min(c["top_k"], -(-n // BLOCK)) - 1) * BLOCK + (n - 1) % BLOCK + 1) for n in lens)
    groups = max(c["Hp"], c["Hkv"])
    return {"bytes": seen * groups * 2 * row + sum(lens) * 256 + new, "flops": 4 * D * seen * c["Hq"] + 2 * D * sum(lens) * c["Hp"]}


# ------------------------------------------------------------------------------------------ inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)

    s = {"case": c, "scale": D ** -0.5}
    if c["op"] in ("axes", "axes_append"):
        heads, n = _heads(c), c.get("S", 1)
        x = randn(c["B"], n, sum(heads), D)
        x *= torch.exp(0.5 * torch.randn((c["B"], n, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)
        s["x"], s["heads"], s["axes"] = x, heads, _axes(c)
        w = lambda: 1 + 0.1 * torch.randn(D, generator=g, device="cuda")  # noqa: E731
        s["weights"] = [w(), w(), None, w(), w()]  # v goes through as it is
        s["rotate"] = [True, True, False, True, True]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
        # frames of 24 x 40 patches: time counts frames, the other axes rows and columns of a frame
        at = torch.randint(0, 100000, (c["B"], 1), generator=g, device="cuda") + torch.arange(n, device="cuda")
        grid = [at // 960, at // 40 % 24, at % 40, at]
        s["positions"] = torch.stack(grid[:c["A"]]).to(torch.int32).contiguous()
        if c["op"] == "axes":
            s["dy"] = [randn(c["B"], n, h, D) for h in heads]
        else:
            s["seq_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
            s["caches"] = [None] + [randn(c["B"], c["cap"], h, D) for h in heads[1:3]] + [None, randn(c["B"], c["cap"], 1, D)]
        return s
    if c["op"] == "packed":
        s["lengths"] = _documents(c)
        s["q"], s["dout"] = randn(c["T"], c["Hq"], D), randn(c["T"], c["Hq"], D)
        s["k"], s["v"] = (randn(c["T"], c["Hkv"], D) for _ in range(2))
        return s
    rows = (c["B"], c["Hkv"], c["cap"] // BLOCK, BLOCK, D)
    if c["op"] == "store":
        s["k"], s["v"] = (randn(c["B"], c["N"], c["Hkv"], D) for _ in range(2))
        s["v"] *= 0.05  # values are not normed
        s["seq_len"] = torch.full((c["B"],), c["N"], dtype=torch.int32, device="cuda")
        s["k_cache"], s["v_cache"] = (torch.zeros(rows[:3] + (CHUNK,), dtype=torch.uint8, device="cuda") for _ in range(2))
        return s
    s["q"] = randn(c["B"], c["Hq"], D)
    s["k"], s["v"] = randn(c["B"], 1, c["Hkv"], D), randn(c["B"], 1, c["Hkv"], D, scale=0.5)
    s["k_cache"], s["v_cache"] = _pack(_codes(randn(*rows))), _pack(_codes(randn(*rows, scale=0.5)))
    s["seq_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    if c["op"] == "sparse":
        # in steps of a quarter, so that every order of summation gives the same scores and the selection is one
        quarter = lambda *shape: ((torch.randn(shape, generator=g, device="cuda") * 4).round() / 4).to(torch.bfloat16)  # noqa: E731
        s["qp"], s["kp"], s["kp_cache"] = quarter(c["B"], c["Hp"], D), quarter(c["B"], 1, 1, D), quarter(c["B"], c["cap"], 1, D)
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


def _axes_plain(s):
    c = s["case"]
    eps, rot, inter = 1e-6, c["rot"], c["inter"]
    a = s["positions"].double()[s["axes"]].permute(1, 2, 0) * s["inv_freq"].double()  # far positions: 32 bits lose the angle
    cos, sin = a.cos().float().unsqueeze(-2), a.sin().float().unsqueeze(-2)
    xs = s["x"].split(s["heads"], 2)
    ys = [_norm_rope_plain(x, w, r, cos, sin, rot, inter, eps) for x, w, r in zip(xs, s["weights"], s["rotate"])]
    if c["op"] == "axes_append":
        b, row = torch.arange(c["B"], device="cuda").view(-1, 1), s["seq_len"].long().view(-1, 1) - 1
        return [y if cache is None else cache.index_put_((b, row), y) for y, cache in zip(ys, s["caches"])]
    back = [_norm_rope_back_plain(x, w, dy, r, cos, sin, rot, inter, eps)
            for x, w, dy, r in zip(xs, s["weights"], s["dy"], s["rotate"])]
    return ys, torch.cat([b[0] for b in back], 2), [b[1] for b in back if b[1] is not None]


def _packed_plain(s):
    """Blocks of bs queries, each against the keys that its first query's window or sequence begins with."""
    c, scale = s["case"], s["scale"]
    T, Hkv, G = c["T"], c["Hkv"], c["Hq"] // c["Hkv"]
    dev = s["q"].device
    lens = torch.tensor(s["lengths"] + [c["pad"]], device=dev)
    ends = lens.cumsum(0)
    starts = torch.repeat_interleave(ends - lens, lens)  # of each token's sequence
    N, span = T - c["pad"], min(_window(c), max(s["lengths"]))
    bs = min(256, T)
    nb = -(-T // bs)
    t = torch.arange(nb * bs, device=dev).view(nb, bs)
    j = t[:, :1] - (span - 1) + torch.arange(span - 1 + bs, device=dev)
    tc, jc = t.clamp(max=T - 1), j.clamp(0, T - 1)
    lo = torch.maximum(starts[tc], tc - (span - 1))
    seen = (j[:, None] <= t[..., None]) & (j[:, None] >= lo[..., None]) & (t[..., None] < N)
    qb = s["q"].float()[tc].view(nb, bs, Hkv, G, D)
    kb, vb = s["k"].float()[jc], s["v"].float()[jc]
    sc = torch.einsum("nthgd,njhd->nhgtj", qb, kb).mul_(scale).masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_(min=-1e30)  # rows behind the last sequence see nothing
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p.div_(l.clamp(min=1e-30))
    ob = torch.einsum("nhgtj,njhd->nhgtd", p, vb)
    rows = lambda x: x.permute(0, 3, 1, 2, 4).flatten(0, 1)[:T].flatten(1, 2)  # noqa: E731
    half = lambda x: x.to(torch.bfloat16).contiguous()  # noqa: E731
    o = rows(ob)
    lse = rows(torch.where(l > 0, m + l.log(), -math.inf)).squeeze(-1).t().contiguous()
    if not c["train"]:
        return half(o), lse
    dob = s["dout"].float()[tc].view(nb, bs, Hkv, G, D) * (t < N).view(nb, bs, 1, 1, 1)
    dv = torch.zeros(s["v"].shape, dtype=torch.float32, device=dev)
    dk = torch.zeros_like(dv)
    at = jc.flatten()
    dv.index_add_(0, at, torch.einsum("nhgtj,nthgd->njhd", p, dob).flatten(0, 1))
    ds = torch.einsum("nthgd,njhd->nhgtj", dob, vb)
    ds.sub_((dob.permute(0, 2, 3, 1, 4) * ob).sum(-1, keepdim=True)).mul_(p)
    dq = rows(torch.einsum("nhgtj,njhd->nhgtd", ds, kb)) * scale
    dk.index_add_(0, at, torch.einsum("nhgtj,nthgd->njhd", ds, qb).flatten(0, 1))
    return half(o), lse, half(dq), half(dk * scale), half(dv)


def _codes(x):
    """Rows x [..., 128] in 4 bits: (codes [..., 128], scales as bytes [..., 8], exponents + 127 [...]), all uint8."""
    x = x.float()
    top = x.abs().amax(-1) / 6
    e = (torch.frexp(top).exponent - 8).clamp_(E_MIN, E_MAX)  # top 2^-e in [128, 256)
    e = torch.where(top > 0, e, E_MIN)
    y = torch.ldexp(x, -e.unsqueeze(-1)).unflatten(-1, (D // 16, 16))
    scale = (y.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    f = scale.float().unsqueeze(-1)
    r = torch.where(f > 0, y.abs() / f, 0)
    code = (r > 0.25).byte() + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5)  # ties to even
    return (code + 8 * (y < 0)).flatten(-2).byte(), scale.view(torch.uint8), (e + 127).byte()


def _pack(parts):
    """Blocks [..., 128 rows] of codes, scales and exponents as bytes [..., CHUNK]."""
    code, scale, e = parts
    return torch.cat([(code[..., 0::2] | code[..., 1::2] << 4).flatten(-2), scale.flatten(-2), e], -1)


def _put(cache, x, first):
    """Writes rows x [B, N, H, 128] to the positions first[b] .. of a packed cache."""
    code, scale, e = _codes(x)
    B, N, H, _ = x.shape
    pos = first.view(B, 1, 1) + torch.arange(N, device=x.device).view(1, N, 1)
    b, h = torch.arange(B, device=x.device).view(B, 1, 1), torch.arange(H, device=x.device).view(1, 1, H)
    blk, row = pos // BLOCK, pos % BLOCK
    cache[..., :BLOCK * 64].unflatten(-1, (BLOCK, 64))[b, h, blk, row] = code[..., 0::2] | code[..., 1::2] << 4
    cache[..., BLOCK * 64:BLOCK * 72].unflatten(-1, (BLOCK, 8))[b, h, blk, row] = scale
    cache[..., BLOCK * 72:][b, h, blk, row] = e


def _values(cache):
    """The fp32 values [B, H, rows, 128] that a packed cache [B, H, blocks, CHUNK] stands for."""
    code = cache[..., :BLOCK * 64].unflatten(-1, (BLOCK, 64))
    code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=cache.device)
    x = grid[code.int()].unflatten(-1, (D // 16, 16))
    x.mul_(cache[..., BLOCK * 64:BLOCK * 72].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, 8)).unsqueeze(-1))
    x = x.flatten(-2)
    return torch.ldexp(x, cache[..., BLOCK * 72:].int().sub(127).unsqueeze(-1)).flatten(2, 3)


def _attend_plain(s, seen):
    """softmax(scale q K^T) V over the keys `seen` [B, groups, cap], the query heads of a group together."""
    c = s["case"]
    B, groups = c["B"], seen.shape[1]
    k, v = (_values(s[x]).repeat_interleave(groups // c["Hkv"], 1) for x in ("k_cache", "v_cache"))
    q = s["q"].float().view(B, groups, -1, D)
    sc = torch.einsum("bhgd,bhjd->bhgj", q, k) * s["scale"]
    sc = sc.masked_fill_(~seen[:, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgj,bhjd->bhgd", p / l, v)
    return o.reshape(B, c["Hq"], D).to(torch.bfloat16), (m + l.log()).reshape(B, c["Hq"])


def _select_plain(s):
    """The key blocks of each proxy head [B, Hp, top_k], -1 padded, and the keys of them up to the newest token."""
    c, n = s["case"], s["seq_len"].long()
    blocks, last = c["cap"] // BLOCK, (n - 1) // BLOCK
    best = torch.einsum("bpd,bjd->bpj", s["qp"].float(), s["kp_cache"].float().squeeze(2))
    best = best.unflatten(-1, (blocks, BLOCK)).amax(-1)
    i = torch.arange(blocks, device=n.device)
    best = best.masked_fill(i >= last[:, None, None], -math.inf).masked_fill(i == last[:, None, None], math.inf)
    order = torch.sort(best, dim=-1, descending=True, stable=True).indices[..., :c["top_k"]]  # ties to the lower block
    taken = torch.zeros_like(best, dtype=torch.bool).scatter_(-1, order, True) & (i <= last[:, None, None])
    idx = torch.where(taken, i, blocks).sort(-1).values
    idx = torch.nn.functional.pad(idx, (0, max(0, c["top_k"] - blocks)), value=blocks)[..., :c["top_k"]]
    j = torch.arange(c["cap"], device=n.device)
    return torch.where(idx < blocks, idx, -1).int(), taken.repeat_interleave(BLOCK, -1) & (j < n[:, None, None])


def _q4_plain(s):
    c = s["case"]
    n = s["seq_len"].long()
    first = n - s["k"].shape[1]
    _put(s["k_cache"], s["k"], first)
    _put(s["v_cache"], s["v"], first)
    if c["op"] == "store":
        return [_values(s[x])[:, :, :c["N"]].transpose(1, 2).to(torch.bfloat16).contiguous() for x in ("k_cache", "v_cache")]
    if c["op"] == "step":
        j, n = torch.arange(c["cap"], device=n.device), n.view(-1, 1)
        seen = (j < n) & ((j >= n - c["W"]) | (j < c["sinks"]))
        return _attend_plain(s, seen[:, None].expand(-1, c["Hkv"], -1))
    s["kp_cache"][torch.arange(c["B"], device=n.device), n - 1] = s["kp"].squeeze(1)
    idx, seen = _select_plain(s)
    return _attend_plain(s, seen.repeat_interleave(max(c["Hp"], c["Hkv"]) // c["Hp"], 1)) + (idx,)


def run(s):
    c = s["case"]
    if not own:
        return _axes_plain(s) if "axes" in s else _packed_plain(s) if c["op"] == "packed" else _q4_plain(s)
    from block_sparse_attention_qp_gb300 import binding as msa
    if "axes" in s:
        xs = s["x"].split(s["heads"], 2)
        how = dict(positions=s["positions"], rotate=s["rotate"], interleaved=c["inter"], axes=s["axes"])
        if c["op"] == "axes_append":
            return msa.msa_norm_rope_append(xs, s["weights"], s["inv_freq"], s["seq_len"], s["caches"], **how)
        ys = msa.msa_norm_rope_forward(xs, s["weights"], s["inv_freq"], **how)
        dx = torch.empty_like(s["x"])
        _, dws = msa.msa_norm_rope_backward(xs, s["weights"], s["dy"], s["inv_freq"], dxs=dx.split(s["heads"], 2), **how)
        return list(ys), dx, [d for d in dws if d is not None]
    if c["op"] == "packed":
        plan = msa.msa_packed_plan(s["lengths"], c["Hq"], c["Hkv"], rows=c["T"], window=c["W"] or None, device=s["q"].device)
        o, lse = msa.msa_packed_forward(s["q"], s["k"], s["v"], plan, s["scale"])
        if not c["train"]:
            return o, lse
        return (o, lse) + msa.msa_packed_backward(s["q"], s["k"], s["v"], o, lse, s["dout"], plan, s["scale"])
    if c["op"] == "sparse":
        msa.msa_norm_rope_append([s["k"], s["v"], s["kp"]], None, None, s["seq_len"], [s["k_cache"], s["v_cache"], s["kp_cache"]])
        return msa.msa_decode_q4(s["q"], s["qp"], s["k_cache"], s["v_cache"], s["kp_cache"], s["seq_len"], c["top_k"], s["scale"])
    msa.msa_norm_rope_append([s["k"], s["v"]], None, None, s["seq_len"], [s["k_cache"], s["v_cache"]])
    if c["op"] == "store":
        return [msa.msa_q4_read(s[x], 0, c["N"]) for x in ("k_cache", "v_cache")]
    return msa.msa_window_decode_q4(s["q"], s["k_cache"], s["v_cache"], s["seq_len"], c["W"], c["sinks"], s["scale"])


# ------------------------------------------------------------------------------------------ exact values
def _exact_axes(s):
    """Rotation as a complex product, gradients from the derivative of x / rms(x), a token chunk at a time."""
    c = s["case"]
    rot, inter, eps = c["rot"], c["inter"], 1e-6
    f, axis = s["inv_freq"].double(), torch.tensor(s["axes"], device="cuda")

    def turn(u, a, z, sign):
        x = u[..., :rot].unflatten(-1, (rot // 2, 2)) if inter else u[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        x = torch.view_as_complex(x.contiguous())
        ang = s["positions"][:, :, a:z].double().index_select(0, axis).movedim(0, -1)[:, :, None] * f
        x = torch.view_as_real(x * torch.polar(torch.ones_like(ang), sign * ang))
        x = x.flatten(-2) if inter else x.transpose(-1, -2).flatten(-2)
        return torch.cat([x, u[..., rot:]], -1)

    ys, dxs, dws, at = [], [], [], 0
    for i, h in enumerate(s["heads"]):
        x, w = s["x"][:, :, at:at + h], s["weights"][i]
        at += h
        y, dx = torch.empty(x.shape, dtype=torch.float64, device="cuda"), torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(D, dtype=torch.float64, device="cuda")
        for a in range(0, x.shape[1], 4096):
            z = min(a + 4096, x.shape[1])
            xc = x[:, a:z].double()
            rms = (xc.pow(2).sum(-1, keepdim=True) / D + eps).sqrt()
            u = xc if w is None else xc / rms * w.double()
            y[:, a:z] = turn(u, a, z, 1) if s["rotate"][i] else u
            if c["op"] == "axes":
                gr = s["dy"][i][:, a:z].double()
                gr = turn(gr, a, z, -1) if s["rotate"][i] else gr
                if w is not None:
                    dw += (gr * xc / rms).sum((0, 1, 2))
                    gr = gr * w.double()
                    gr = gr / rms - xc * (gr * xc).sum(-1, keepdim=True) / (D * rms ** 3)
                dx[:, a:z] = gr
        if c["op"] == "axes_append" and s["caches"][i] is not None:
            full = s["caches"][i].double()
            for b, n in enumerate(s["seq_len"].tolist()):
                full[b, n - 1] = y[b, 0]
            y = full
        ys.append(y)
        dxs.append(dx)
        if w is not None:
            dws.append(dw)
    return ys if c["op"] == "axes_append" else (ys, torch.cat(dxs, 2), dws)


def _exact_packed(s):
    """One sequence, KV head and run of queries at a time, from the definition."""
    c, scale = s["case"], s["scale"]
    G, W = c["Hq"] // c["Hkv"], _window(c)
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, dq, dk, dv = zero(s["q"]), zero(s["q"]), zero(s["k"]), zero(s["v"])
    lse = torch.full((c["Hq"], c["T"]), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for n in s["lengths"]:
        for a in range(0, n, 1024):
            z = min(n, a + 1024)
            lo = max(0, a - W + 1)
            diff = torch.arange(a, z, device="cuda")[:, None] - torch.arange(lo, z, device="cuda")
            hidden = (diff < 0) | (diff >= W)
            qs, ks = slice(at + a, at + z), slice(at + lo, at + z)
            for h in range(c["Hkv"]):
                hs = slice(h * G, h * G + G)
                q, k, v = s["q"][qs, hs].double().transpose(0, 1), s["k"][ks, h].double(), s["v"][ks, h].double()
                sc = (q @ k.T * scale).masked_fill_(hidden, -math.inf)
                ls = sc.logsumexp(-1, keepdim=True)
                p = (sc - ls).exp()
                ob = p @ v
                o[qs, hs], lse[hs, qs] = ob.transpose(0, 1), ls[..., 0]
                if c["train"]:
                    do = s["dout"][qs, hs].double().transpose(0, 1)
                    ds = p * (do @ v.T - (do * ob).sum(-1, keepdim=True)) * scale
                    dq[qs, hs] = (ds @ k).transpose(0, 1)
                    dk[ks, h] += torch.einsum("gtj,gtd->jd", ds, q)
                    dv[ks, h] += torch.einsum("gtj,gtd->jd", p, do)
        at += n
    return (o, lse, dq, dk, dv) if c["train"] else (o, lse)


def _exact_row(x):
    """The 64-bit values that rows x [..., 128] keep in 4 bits, by the nearest members of the two grids."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True) / 6
    e = torch.where(top > 0, torch.floor(torch.log2(top)) - 7, E_MIN).clamp(E_MIN, E_MAX)
    y = (x * torch.exp2(-e)).unflatten(-1, (D // 16, 16))

    def nearest(v, grid):  # members ascending; of two equally near the one at an even place
        g = torch.tensor(grid, dtype=torch.float64, device=v.device)
        i = torch.searchsorted(g, v.contiguous()).clamp(1, len(grid) - 1)
        below, above = v - g[i - 1], g[i] - v
        return g[torch.where((below < above) | ((below == above) & (i % 2 == 1)), i - 1, i)]

    fine = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** p for p in range(-6, 9) for m in range(8)][:119]
    s = nearest(y.abs().amax(-1, keepdim=True) / 6, fine)
    r = nearest(torch.where(s > 0, y.abs() / s, 0), [0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return (r * s * y.sign()).flatten(-2) * torch.exp2(e)


def _exact_q4(s):
    c = s["case"]
    if c["op"] == "store":
        return [_exact_row(s["k"]), _exact_row(s["v"])]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((c["B"], c["Hq"]), dtype=torch.float64, device="cuda")
    groups = max(c.get("Hp", 1), c["Hkv"]) if c["op"] == "sparse" else c["Hkv"]
    G = c["Hq"] // groups
    for b, n in enumerate(s["seq_len"].tolist()):
        k, v = (_values(s[x][b:b + 1])[0].double() for x in ("k_cache", "v_cache"))
        k[:, n - 1], v[:, n - 1] = _exact_row(s["k"][b, 0]), _exact_row(s["v"][b, 0])
        if c["op"] == "sparse":
            kp = s["kp_cache"][b, :n, 0].double()
            kp[n - 1] = s["kp"][b, 0, 0].double()
            z = s["qp"][b].double() @ kp.T
        for a in range(groups):
            if c["op"] == "step":
                lo = max(0, n - c["W"])
                j = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, n, device="cuda")])
            else:
                zp = z[a * c["Hp"] // groups]
                own_block = (n - 1) // BLOCK
                best = [(-float(zp[i * BLOCK:(i + 1) * BLOCK].max()), i) for i in range(own_block)]
                blocks = sorted([own_block] + [i for _, i in sorted(best)[:c["top_k"] - 1]])
                j = torch.cat([torch.arange(i * BLOCK, min(n, (i + 1) * BLOCK), device="cuda") for i in blocks])
            kv, hs = a * c["Hkv"] // groups, slice(a * G, a * G + G)
            sc = s["q"][b, hs].double() @ k[kv, j].T * s["scale"]
            lse[b, hs] = sc.logsumexp(-1)
            o[b, hs] = sc.softmax(-1) @ v[kv, j]
    return (o, lse) if c["op"] == "step" else (o, lse, None)


def exact(c, seed):
    s = prepare(c, seed)
    return _exact_axes(s) if "axes" in s else _exact_packed(s) if c["op"] == "packed" else _exact_q4(s)
