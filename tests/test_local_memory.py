"""Which memory the tensors of one norm-and-rotation call may share: the check on the host against the bytes
themselves, and the refusals a user meets."""
import ctypes
import itertools
import random

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build

P = ctypes.c_void_p
A = P(0x10000)  # aligned, never dereferenced: every call here fails on the host
NULL = P(0)
CLASH = b"same output"
INPUT = b"overlaps an input"


@pytest.fixture(scope="module")
def lib():
    return msa.load_library(build.build())


def units(at, B, sb, N, st, heads):
    """The 16-byte units of a tensor's rows (strides in elements)."""
    return {at // 16 + (b * sb + n * st) // 8 + i for b in range(B) for n in range(N) for i in range(16 * heads)}


def refusal(lib, op, s, parts):
    """What the library says of a call: None where nothing but the last check (a workspace of no bytes) refuses it."""
    arr = (msa.RopePart * len(parts))(*parts)
    if op == "append":
        rc = lib.msa_norm_rope_append(ctypes.byref(s), arr, len(parts), A, NULL, A, 0, NULL)
    else:
        rc = lib.msa_norm_rope_backward(ctypes.byref(s), arr, len(parts), NULL, NULL, A, 0, NULL)
    assert rc in (1, 3), (rc, lib.msa_last_error())
    return None if rc == 3 else lib.msa_last_error()


def test_backward_outputs_by_their_bytes(lib):
    """Random slices of a small arena: refused exactly where bytes are shared that may not be."""
    rng = random.Random(5)
    seen = {None: 0, CLASH: 0, INPUT: 0}
    for _ in range(4000):
        B, N = rng.choice([1, 2, 3]), rng.choice([1, 2, 4])
        s = msa.RopeShape(B, N, 128, 0, 0, 0, 1e-6)
        heads = [rng.choice([1, 2, 3]) for _ in range(2)]
        wide = rng.choice([4, 6, 9]) * 128  # a token of the arena
        tensors = {}
        for i, name in itertools.product(range(2), ("x", "dy", "dx")):
            first, second = rng.choice([(wide * N, wide), (wide, wide * B), (heads[i] * 128 * N, heads[i] * 128)])
            base = 0x100000 * rng.choice([1, 1, 2, 3, 4]) + 256 * rng.randrange(24) + rng.choice([0, 0, 16])
            tensors[i, name] = (base, first if B > 1 else 0, second if N > 1 else 0)
        if rng.random() < 0.3:
            tensors[1, "dx"] = tensors[1, rng.choice(["x", "dy"])]
        cover = {k: units(t[0], B, t[1], N, t[2], heads[k[0]]) for k, t in tensors.items()}
        want = set()
        for i in range(2):
            if len(cover[i, "dx"]) < 16 * heads[i] * B * N:
                want.add(b"strides are too small")
            for k, c in cover.items():
                if k == (i, "dx") or not c & cover[i, "dx"]:
                    continue
                if k[1] == "dx":
                    want.add(CLASH)
                elif k[0] != i or tensors[k] != tensors[i, "dx"]:
                    want.add(INPUT)
        parts = [msa.RopePart(*tensors[i, "x"], *tensors[i, "dy"], *tensors[i, "dx"], 0, 0, heads[i], 0) for i in range(2)]
        got = refusal(lib, "backward", s, parts)
        if got is None:
            assert not want, (tensors, heads, B, N)
            seen[None] += 1
        elif b"strides" in got:  # strides that do not nest are refused whether or not rows meet
            continue
        else:
            assert any(w in got for w in want), (got, want, tensors, heads, B, N)
            seen[CLASH if CLASH in got else INPUT] += 1
    assert min(seen.values()) > 100, seen  # each kind is met


def test_append_outputs(lib):
    """Caches as slices of one buffer, with strides of their own, that meet, that meet an x."""
    s = msa.RopeShape(2, 3, 128, 0, 0, 16, 1e-6)
    x = (0x10000, 3 * 256, 256)

    def part(y, x=x, heads=2, cache=True):
        return msa.RopePart(*x, *y, 0, 0, 0, 0, 0, heads, msa.ROPE_CACHE if cache else 0)

    wide = 5 * 128  # k, v and one proxy head of a token side by side
    k, v, p = ((0x100000 + 256 * h, 16 * wide, wide) for h in (0, 2, 4))
    assert refusal(lib, "append", s, [part(k), part(v), part(p, heads=1)]) is None
    assert CLASH in refusal(lib, "append", s, [part(k), part((0x100000 + 256, 16 * wide, wide))])
    assert CLASH in refusal(lib, "append", s, [part(k), part(v, heads=3), part(p, heads=1)])
    # one buffer a sequence, the tensors one after the other in it: other strides, no shared bytes
    each = 16 * 5 * 128
    k, v, p = (0x100000, each, 256), (0x100000 + 16 * 512, each, 256), (0x100000 + 32 * 512, each, 128)
    assert refusal(lib, "append", s, [part(k), part(v), part(p, heads=1)]) is None
    assert CLASH in refusal(lib, "append", s, [part(k), part(v), part((p[0] - 256, each, 128), heads=1)])
    # the cache's last row counts, not the tokens of the call
    end = 0x200000 + (16 + 15) * 512
    assert CLASH in refusal(lib, "append", s, [part((0x200000, 16 * 256, 256)), part((end, 768, 256), cache=False)])
    assert refusal(lib, "append", s, [part((0x200000, 16 * 256, 256)), part((end + 512, 768, 256), cache=False)]) is None
    # an x inside a cache, its own or another's
    inside = (0x100000 + 512, 16 * 256, 256)
    assert INPUT in refusal(lib, "append", s, [part((0x100000, 16 * 256, 256), x=inside)])
    assert INPUT in refusal(lib, "append", s, [part((0x100000, 16 * 256, 256)), part((0x300000, 16 * 256, 256), x=inside)])
    # rows of one output that meet, and a plain output in the rows of its x
    assert b"too small" in refusal(lib, "append", s, [part((0x100000, 16 * 256, 128))])
    assert refusal(lib, "append", s, [part(x, cache=False)]) is None
    assert INPUT in refusal(lib, "append", s, [part((x[0] + 256, x[1], x[2]), cache=False)])


def test_weight_gradients_that_meet(lib):
    s = msa.RopeShape(1, 4, 128, 0, 0, 0, 1e-6)
    row = lambda at: (at, 0, 256)  # noqa: E731
    part = lambda i, dw: msa.RopePart(*row(0x10000 + 0x1000 * i), *row(0x20000 + 0x1000 * i), *row(0x30000 + 0x1000 * i),  # noqa: E731
                                      0x50000, dw, 2, 0)
    assert refusal(lib, "backward", s, [part(0, 0x60000), part(1, 0x60000 + 512)]) is None
    for d in (0, 16, 496, -496):
        assert CLASH in refusal(lib, "backward", s, [part(0, 0x60000), part(1, 0x60000 + d)])


@pytest.mark.gpu
def test_refused_through_the_binding():
    dev = "cuda:0"
    x = torch.randn(2, 5, 4, 128, device=dev).to(torch.bfloat16)
    xs = x.split((2, 2), 2)
    dys = [torch.randn(2, 5, 2, 128, device=dev).to(torch.bfloat16) for _ in range(2)]
    want, _ = msa.msa_norm_rope_backward(xs, None, dys, None)
    kept = [d.clone() for d in dys]
    for dxs in (dys[::-1], [x[:, :, :2], x[:, :, 1:3]], [x[:, :, 2:], dys[1]]):
        with pytest.raises(msa.MSAError, match="overlap"):
            msa.msa_norm_rope_backward(xs, None, dys, None, dxs=dxs)
    assert all(torch.equal(a, b) for a, b in zip(dys, kept))
    got, _ = msa.msa_norm_rope_backward(xs, None, dys, None, dxs=list(x.clone().split((2, 2), 2)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got, _ = msa.msa_norm_rope_backward(xs, None, [d.clone() for d in dys], None, dxs=xs)  # in place of x
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    arena = torch.zeros(2, 64, 5, 128, dtype=torch.bfloat16, device=dev)
    n = torch.tensor([5, 64], dtype=torch.int32, device=dev)
    with pytest.raises(msa.MSAError, match="overlap"):
        msa.msa_norm_rope_append([w.contiguous() for w in want], None, None, n, [arena[:, :, :2], arena[:, :, 1:3]])
    assert not arena.any()
    msa.msa_norm_rope_append(want, None, None, n, [arena[:, :, :2], arena[:, :, 2:4]])
    assert torch.equal(arena[0, :5, :4], torch.cat(want, 2)[0]) and torch.equal(arena[1, 59:, :4], torch.cat(want, 2)[1])
    assert not arena[:, :, 4].any() and not arena[0, 5:].any() and not arena[1, :59].any()
