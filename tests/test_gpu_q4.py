"""Caches in 4 bits on the GPU: what is stored, bit for bit, and the decode steps that read them."""
import ctypes
import random

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_q4 as plain
from tests.plain_local import check

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(torch.bfloat16)


def lens32(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def same_rows(cache, rows, want):
    """Rows `rows` of every head are those of the bf16 rows `want` [B, n, H, 128]."""
    got, exp = plain.unpack(cache), plain.quantise(want)
    for name, a, b in zip(("exponents", "scales", "codes"), reversed(got), reversed(exp)):
        a = torch.stack([a[i, r] for i, r in enumerate(rows)])
        if name == "codes":  # -0 is 0
            a = torch.where(a == 8, 0, a)
        assert torch.equal(a, b), f"{name}: {int((a != b).sum())} differ"


@pytest.mark.parametrize("B,N,H,cap,lens", [
    (1, 1, 1, 128, [1]), (1, 1, 1, 128, [128]), (3, 1, 2, 256, [1, 129, 256]), (2, 5, 8, 384, [5, 300]),
    (1, 300, 3, 384, [301]), (2, 999, 2, 1024, [1000, 1024]), (128, 1, 8, 256, [1 + i * 2 for i in range(128)]),
])
def test_stored_rows(B, N, H, cap, lens):
    r = gen(1)
    x = r(B, N, H, 128) * torch.exp2(torch.randint(-30, 30, (B, N, H, 1), device="cuda").float()).to(torch.bfloat16)
    x *= torch.exp2(torch.randint(-9, 2, (B, N, H, 8, 1), device="cuda").float()).repeat_interleave(16, -1).flatten(-2).to(torch.bfloat16)
    cache = msa.msa_q4_cache(B, H, cap, "cuda")
    cache.random_(0, 256)
    before = cache.clone()
    out, = msa.msa_norm_rope_append([x], None, None, lens32(*lens), [cache])
    assert out is cache
    rows = [torch.arange(n - N, n, device="cuda") for n in lens]
    same_rows(cache, rows, x)
    other = [plain.unpack(c) for c in (before, cache)]
    for a, b in zip(*other):
        for i, n in enumerate(lens):
            keep = torch.ones(cap, dtype=torch.bool, device="cuda")
            keep[n - N:n] = False
            assert torch.equal(a[i, keep], b[i, keep])
    want = plain.values(plain.unpack(cache))
    for i, n in enumerate(lens):  # (the other rows' bytes are no rows of the format)
        assert (msa.msa_q4_read(cache, n - N, N)[i].double() == want[i, n - N:n]).all()


def test_stored_extremes():
    """Zeros, a single value, borders between two codes and two scales, the ends of the exponents, values that are not finite."""
    x = torch.zeros(1, 16, 1, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 1, 0, 77] = -3.0
    x[0, 2, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6] + [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6.0])
    x[0, 3] = x[0, 2] * 2.0 ** -60
    x[0, 4, 0] = torch.arange(128) * 2.0 ** -110
    x[0, 5, 0] = torch.arange(128) * 2.0 ** -133
    x[0, 6, 0] = torch.arange(128) * 2.0 ** 80
    x[0, 7, 0] = 3e38
    x[0, 8, 0, 5] = float("inf")
    x[0, 9, 0, 100] = float("nan")
    x[0, 10, 0, 0], x[0, 10, 0, 16] = 1.0, 2.0 ** -13  # a scale that just has all its bits
    x[0, 11, 0, 0], x[0, 11, 0, 16] = 1.0, 2.0 ** -19  # one that is rounded away
    x[0, 12, 0] = -(1 + torch.arange(128) / 128) * 6
    x[0, 13, 0, ::16] = 6 * (1 + (2 * torch.arange(8) + 1) / 16).to(torch.bfloat16).cuda()  # between two scales
    x[0, 14] = -0.0
    x[0, 15, 0, 3], x[0, 15, 0, 60] = -float("inf"), 1.0
    cache = msa.msa_q4_cache(1, 1, 128, "cuda")
    msa.msa_norm_rope_append([x], None, None, lens32(16), [cache])
    same_rows(cache, [torch.arange(16, device="cuda")], x)
    got = msa.msa_q4_read(cache, 0, 16)[0, :, 0].double()
    nan = torch.isnan(got).all(-1)
    assert nan.tolist() == [i in (8, 9, 15) for i in range(16)]
    assert torch.isfinite(got[~nan]).all()


def test_stored_beside_others():
    """k normed and rotated, v as it is, from the slices of one projection: what goes to the caches in 4 bits is what a
    bf16 output of the same call holds, and a bf16 cache beside them is written too."""
    r = gen(2)
    B, N, Hq, H = 3, 4, 8, 2
    x = r(B, N, Hq + 3 * H + 1, 128)
    q, k, v, k2, kp = x.split([Hq, H, H, H, 1], 2)
    k2.copy_(k)
    w = 1 + 0.1 * torch.randn(128, device="cuda")
    freq = 10000.0 ** (-torch.arange(0, 128, 2, device="cuda") / 128)
    n = lens32(4, 130, 256)
    kc, vc = (msa.msa_q4_cache(B, H, 256, "cuda") for _ in range(2))
    kpc = torch.zeros(B, 256, 1, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    yq, _, _, yk, _ = msa.msa_norm_rope_append([q, k, v, k2, kp], [w, w, None, w, w], freq, n, [None, kc, vc, None, kpc],
                                               rotate=[True, True, False, True, True], ws=ws)
    assert msa.msa_device_status(ws) == 0
    rows = [torch.arange(m - N, m, device="cuda") for m in n.tolist()]
    same_rows(kc, rows, yk)
    same_rows(vc, rows, v)
    plain_q, plain_kp = msa.msa_norm_rope_append([q, kp], [w, w], freq, n, [None, torch.zeros_like(kpc)])
    # (another instance of the kernel: the same roundings up to the contraction of a product and a sum)
    assert (yq.float() - plain_q.float()).abs().max() <= 2 ** -7 * plain_q.float().abs().max()
    assert (kpc.float() - plain_kp.float()).abs().max() <= 2 ** -7 * plain_kp.float().abs().max()


def test_lengths_out_of_range_store_nothing():
    cache = msa.msa_q4_cache(4, 2, 128, "cuda").fill_(17)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    x = gen(3)(4, 2, 2, 128)
    msa.msa_norm_rope_append([x], None, None, lens32(1, 129, 2, -5), [cache], ws=ws)
    assert msa.msa_device_status(ws) == 1
    assert (cache[[0, 1, 3]] == 17).all() and not (cache[2] == 17).all()


def filled(r, B, H, cap, lens, scale=1.0, seed=0):
    """K and V caches holding random rows up to lens, bytes of 0xff (scales that are NaN) behind them."""
    caches = []
    for i in range(2):
        c = msa.msa_q4_cache(B, H, cap, "cuda").fill_(255)
        for b, n in enumerate(lens):
            if 1 <= n <= cap:
                msa.msa_norm_rope_append([r(1, n, H, 128, scale=scale if i else 1.0)], None, None, lens32(n), [c[b:b + 1]])
        caches.append(c)
    return caches


def decode_check(q, kc, vc, lens, keys_of, o, lse, cap):
    k, v = (plain.values(plain.unpack(c)) for c in (kc, vc))
    for b, n in enumerate(lens):
        if not 1 <= n <= cap:
            continue
        j = keys_of(b, n)
        want = plain.attend(q[b], k[b, j], v[b, j], SCALE)
        check(f"o[{b}]", o[b], want["o"])
        check(f"lse[{b}]", lse[b], want["lse"])


@pytest.mark.parametrize("Hq,Hkv,cap,lens,W,sinks", [
    (1, 1, 128, [1], 1, 0), (2, 1, 128, [128, 1, 17], 128, 0), (8, 2, 1024, [1, 2, 600, 1024], 128, 4),
    (8, 8, 512, [512, 77], 512, 0), (16, 4, 512, [500], 1, 0), (16, 4, 512, [500], 1, 1), (64, 8, 256, [255, 256], 33, 130),
    (16, 1, 384, [384, 129, 128, 5], 200, 16), (64, 4, 640, [640, 300], 250, 300), (32, 2, 512, [400], 2 ** 31 - 1, 2 ** 31 - 1),
    (8, 1, 8192, [8192, 4000], 8192, 0), (16, 1, 8192, [8191], 5000, 7), (8, 2, 2048, [2048] * 3, 129, 129),
])
def test_window_decode(Hq, Hkv, cap, lens, W, sinks):
    r = gen(Hq * cap + W)
    B = len(lens)
    kc, vc = filled(r, B, Hkv, cap, lens, scale=0.05)
    q = r(B, Hq, 128)
    shape = msa.WindowShape(B, cap, Hq, Hkv, 128, min(W, 2 ** 31 - 1), min(sinks, 2 ** 31 - 1), SCALE)
    ws = torch.full((msa.msa_window_workspace_size(shape, msa.OP_WINDOW_DECODE_Q4),), 255, dtype=torch.uint8, device="cuda")
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(*lens), W, sinks, SCALE, ws=ws)
    assert msa.msa_device_status(ws) == 0
    decode_check(q, kc, vc, lens, lambda b, n: plain.window_keys(n, W, sinks, "cuda"), o, lse, cap)


def test_window_decode_uneven_rows():
    """Values and keys whose magnitudes differ by 2^20 from row to row, queries by head."""
    r = gen(5)
    n, H = 700, 2
    up = lambda *s: torch.exp2(torch.randint(-10, 11, s, device="cuda").float()).to(torch.bfloat16)  # noqa: E731
    kc, vc = (msa.msa_q4_cache(1, H, 768, "cuda") for _ in range(2))
    k, v = r(1, n, H, 128), r(1, n, H, 128)
    k *= torch.exp2(torch.randint(-10, 1, (1, n, H, 1), device="cuda").float()).to(torch.bfloat16)
    v *= up(1, n, H, 1)
    for c, x in ((kc, k), (vc, v)):
        msa.msa_norm_rope_append([x], None, None, lens32(n), [c])
    q = r(1, 8, 128) * torch.exp2(torch.arange(-6, 2, device="cuda").float()).to(torch.bfloat16).view(1, 8, 1)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(n), 700, 0, SCALE)
    decode_check(q, kc, vc, [n], lambda b, m: torch.arange(m, device="cuda"), o, lse, 768)


@pytest.mark.parametrize("zeros", ["all", "the heaviest", "all but one"])
def test_window_decode_values_of_zero(zeros):
    """Rows of zeros have the least exponent, which the weights of their keys are taken relative to."""
    r = gen(12)
    n, H = 5000, 2
    k, v = r(1, n, H, 128, scale=0.5), r(1, n, H, 128)
    if zeros == "all":
        v.zero_()
    elif zeros == "the heaviest":
        k[:, 77] *= 8
        v[:, 77] = 0
    else:
        v[:, :4999] = 0
    caches = [msa.msa_q4_cache(1, H, 5120, "cuda") for _ in range(2)]
    for c, x in zip(caches, (k, v)):
        msa.msa_norm_rope_append([x], None, None, lens32(n), [c])
    q = r(1, 8, 128) * 2
    o, lse = msa.msa_window_decode_q4(q, *caches, lens32(n), n, 0, SCALE)
    decode_check(q, *caches, [n], lambda b, m: torch.arange(m, device="cuda"), o, lse, 5120)
    if zeros == "all":
        assert (o == 0).all()


def test_window_decode_lengths_out_of_range():
    r = gen(6)
    lens, cap = [0, 200, 257, -1, 256], 256
    kc, vc = filled(r, 5, 2, cap, lens)
    q = r(5, 8, 128)
    shape = msa.WindowShape(5, cap, 8, 2, 128, 64, 3, SCALE)
    ws = torch.empty(msa.msa_window_workspace_size(shape, msa.OP_WINDOW_DECODE_Q4), dtype=torch.uint8, device="cuda")
    o = torch.full((5, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8), 3.0, device="cuda")
    rc = msa.load_library().msa_window_decode_q4(ctypes.byref(shape), q.data_ptr(), kc.data_ptr(), vc.data_ptr(), lens32(*lens).data_ptr(),
                                                 o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), msa._stream_of(q.device))
    assert rc == 0 and msa.msa_device_status(ws) == 1
    for b in (0, 2, 3):
        assert (o[b] == 3).all() and (lse[b] == 3).all()
    decode_check(q, kc, vc, lens, lambda b, n: plain.window_keys(n, 64, 3, "cuda"), o, lse, cap)


def test_a_row_that_is_not_finite_shows():
    """... where it is visible, and only there."""
    r = gen(7)
    kc, vc = (msa.msa_q4_cache(2, 1, 256, "cuda") for _ in range(2))
    k, v = r(2, 200, 1, 128), r(2, 200, 1, 128)
    v[1, 150, 0, 3] = float("nan")
    for c, x in ((kc, k), (vc, v)):
        msa.msa_norm_rope_append([x], None, None, lens32(200, 200), [c])
    q = r(2, 4, 128)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(200, 200), 200, 0, SCALE)
    assert torch.isfinite(o[0]).all() and torch.isnan(o[1]).all() and torch.isfinite(lse).all()
    o, _ = msa.msa_window_decode_q4(q, kc, vc, lens32(200, 200), 49, 0, SCALE)
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("Hq,Hkv,Hp,cap,lens,top_k", [
    (8, 2, 2, 512, [1, 128, 129, 512], 2), (64, 8, 8, 2048, [2000, 2048], 4), (16, 4, 1, 1024, [1000, 5], 3),
    (16, 1, 4, 1024, [1024], 16), (16, 1, 1, 640, [600], 5), (8, 8, 8, 512, [257], 1), (32, 2, 2, 8192, [8192], 33),
])
def test_sparse_decode(Hq, Hkv, Hp, cap, lens, top_k):
    r = gen(Hq + Hp + cap)
    B = len(lens)
    kc, vc = filled(r, B, Hkv, cap, lens, scale=0.3)
    q, qp, kp = r(B, Hq, 128), r(B, Hp, 128), r(B, cap, 1, 128)
    n = lens32(*lens)
    ws = torch.full((msa.msa_workspace_size(msa.Shape(B, cap, Hq, Hkv, Hp, 128, top_k, SCALE), msa.OP_DECODE_Q4),), 255,
                    dtype=torch.uint8, device="cuda")
    o, lse, idx = msa.msa_decode_q4(q, qp, kc, vc, kp, n, top_k, SCALE, ws=ws)
    assert msa.msa_device_status(ws) == 0
    kb, vb = (torch.nan_to_num(msa.msa_q4_read(c, 0, cap)) for c in (kc, vc))
    o16, lse16, idx16 = msa.msa_decode(q, qp, kb, vb, kp, n, top_k, SCALE)
    assert torch.equal(idx, idx16)
    k, v = (plain.values(plain.unpack(c)) for c in (kc, vc))
    groups = max(Hp, Hkv)
    G = Hq // groups
    for b, m in enumerate(lens):
        for a in range(groups):
            blocks = [i for i in idx[b, a * Hp // groups].tolist() if i >= 0]
            j = torch.cat([torch.arange(128 * i, min(m, 128 * i + 128), device="cuda") for i in blocks])
            kv, hs = a * Hkv // groups, slice(a * G, a * G + G)
            want = plain.attend(q[b, hs], k[b, j][:, kv:kv + 1], v[b, j][:, kv:kv + 1], SCALE)
            check(f"o[{b}, {a}]", o[b, hs], want["o"])
            check(f"lse[{b}, {a}]", lse[b, hs], want["lse"])


def test_steps_captured_and_on_another_stream():
    """Append and attend, captured once and replayed over new tokens; two graphs of calls with workspaces of their own."""
    r = gen(8)
    B, Hq, H, cap = 2, 8, 2, 256
    kc, vc = filled(r, B, H, cap, [100, 200])
    n = lens32(100, 200)
    q, k, v = r(B, Hq, 128), r(B, 1, H, 128), r(B, 1, H, 128)

    def step():
        msa.msa_norm_rope_append([k, v], None, None, n, [kc, vc])
        return msa.msa_window_decode_q4(q, kc, vc, n, 150, 4, SCALE)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1, stream=side):
            n.add_(1)
            o1, l1 = step()
        with torch.cuda.graph(g2, stream=side):
            o2, l2 = msa.msa_window_decode_q4(q, kc, vc, n, 20, 0, SCALE)
        for i in range(3):
            q.copy_(r(B, Hq, 128))
            k.copy_(r(B, 1, H, 128))
            v.copy_(r(B, 1, H, 128))
            g1.replay()
            g2.replay()
            side.synchronize()
            lens = [101 + i, 201 + i]
            assert n.tolist() == lens
            same_rows(kc, [torch.tensor([m - 1], device="cuda") for m in lens], k)
            decode_check(q, kc, vc, lens, lambda b, m: plain.window_keys(m, 150, 4, "cuda"), o1, l1, cap)
            decode_check(q, kc, vc, lens, lambda b, m: plain.window_keys(m, 20, 0, "cuda"), o2, l2, cap)
    torch.cuda.current_stream().wait_stream(side)


def test_same_bits_every_time():
    r = gen(9)
    kc, vc = filled(r, 2, 2, 4096, [4096, 3000])
    q = r(2, 16, 128)
    a = msa.msa_window_decode_q4(q, kc, vc, lens32(4096, 3000), 4096, 0, SCALE)
    for _ in range(3):
        b = msa.msa_window_decode_q4(q, kc, vc, lens32(4096, 3000), 4096, 0, SCALE)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_cache_past_32_bits():
    """Rows of the last sequence begin behind 2^32 bytes."""
    B, H, cap = 8, 8, 1 << 20
    cache = torch.empty((B, H, cap // 128, msa.Q4_BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32 + 2 ** 29
    r = gen(10)
    n, back = [5, 1, 1, 1, 1, 1, 1, cap], 300
    for m in (cap - back, cap):  # the last 600 rows of the last sequence
        x = r(1, back, H, 128)
        msa.msa_norm_rope_append([x], None, None, lens32(m), [cache[-1:]])
        got = msa.msa_q4_read(cache[-1:], m - back, back)
        assert torch.equal(got.double(), plain.values(plain.quantise(x)))
    msa.msa_norm_rope_append([r(B, 1, H, 128)], None, None, lens32(*n), [cache])
    q = r(B, 16, 128)
    o, lse = msa.msa_window_decode_q4(q, cache, cache, lens32(*n), 500, 0, SCALE)
    kv = msa.msa_q4_read(cache[-1:], cap - 500, 500)[0].double()
    want = plain.attend(q[-1], kv, kv, SCALE)
    check("o", o[-1], want["o"])
    check("lse", lse[-1], want["lse"])


@pytest.mark.parametrize("Hq,H,B,cap", [(8, 8, 64, 1024), (128, 8, 40, 896), (5, 5, 100, 1280), (64, 8, 58, 1024), (470, 470, 1, 128)])
def test_window_decode_of_many_sequences(Hq, H, B, cap):
    """More blocks than stay resident: the long sequences begin first, and each writes its own rows."""
    R = random.Random(B)
    lens = [R.choice([1, cap, cap // 2, R.randint(1, cap), R.randint(1, 200)]) for _ in range(B)]
    test_window_decode(Hq, H, cap, lens, 2 ** 31 - 1, 0)


def test_window_decode_of_many_sequences_with_wrong_lengths():
    r, B, H, cap = gen(23), 64, 8, 1024
    lens = [(i * 97) % cap + 1 for i in range(B)]
    k, v = filled(r, B, H, cap, lens)
    q = r(B, H, 128)
    o, lse = msa.msa_window_decode_q4(q, k, v, lens32(*lens), 2 ** 31 - 1, 0, SCALE)
    for wrong in (0, -1, cap + 1, 2 ** 31 - 1):
        bad = list(lens)
        bad[7] = bad[63] = wrong
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        o2, lse2 = msa.msa_window_decode_q4(q, k, v, lens32(*bad), 2 ** 31 - 1, 0, SCALE, ws=ws)
        assert msa.msa_device_status(ws) == 1
        good = [i for i in range(B) if i not in (7, 63)]
        assert torch.equal(o[good], o2[good]) and torch.equal(lse[good], lse2[good])


@pytest.mark.parametrize("Hq,H,Hp,B,cap,top_k", [(8, 8, 8, 64, 1024, 8), (64, 4, 8, 60, 2048, 6), (32, 4, 2, 116, 1664, 13)])
def test_sparse_decode_of_many_sequences(Hq, H, Hp, B, cap, top_k):
    R = random.Random(B)
    test_sparse_decode(Hq, H, Hp, cap, [R.choice([1, cap, 129, R.randint(1, cap)]) for _ in range(B)], top_k)


@pytest.mark.parametrize("Hq,H,lens,cap,sinks", [(8, 8, [8192, 1, 8191, 4097, 130, 2000], 8192, 0), (32, 2, [12000, 16384, 4096, 5], 16384, 77),
                                                 (4, 4, [1, 3, 100, 6000], 16384, 0)])
def test_window_decode_in_parts(Hq, H, lens, cap, sinks):
    """Several sequences of a large capacity: parts of equal length, most of them of short sequences empty."""
    test_window_decode(Hq, H, cap, lens, 2 ** 31 - 1, sinks)
    test_window_decode(Hq, H, cap, lens, cap - 1000, sinks)
