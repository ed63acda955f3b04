"""Host counts of a packed plan against a walk over every token."""
import ctypes
import random

import pytest

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build


@pytest.fixture(scope="module")
def lib():
    return msa.load_library(build.build())


def table_bytes(lib, lengths, Hq, Hkv, rows, window):
    shape = msa.PackedShape(rows, Hq, Hkv, 128, window)
    return lib.msa_packed_table_bytes(ctypes.byref(shape), (ctypes.c_int32 * max(1, len(lengths)))(*lengths), len(lengths))


def walk(lengths, G, window):
    """(key tiles of 128 tokens, query tiles that see each key block)."""
    lo, hi, at = [], [], 0
    for n in lengths:
        lo += [max(at, at + t - window + 1) for t in range(n)]
        hi += [min(at + n - 1, at + t + window - 1) for t in range(n)]
        at += n
    tt = 128 // G
    tiles = [(hi[min(k + 128, at) - 1] - k) // tt + 1 for k in range(0, at, 128)]
    return at, tiles


@pytest.mark.parametrize("seed", range(12))
def test_counts(lib, seed):
    r = random.Random(seed)
    G, Hkv = r.choice([1, 2, 4, 8, 16]), r.choice([1, 2, 8])
    lengths = [r.choice([0, 1, 2, 127, 128, 129, r.randint(1, 3000)]) for _ in range(r.randint(1, 40))] + [5]
    rows, window = sum(lengths) + r.choice([0, 1, 300]), r.choice([1, 50, 128, 10 ** 6])
    n, tiles = walk(lengths, G, min(window, rows))
    tt, up = 128 // G, lambda x: (x + 255) // 256 * 256  # noqa: E731
    got = table_bytes(lib, lengths, G * Hkv, Hkv, rows, window)
    fixed = 2 * up(4 * n) + up(16 * -(-n // tt)) + up(4 * len(tiles))
    # the rest are the forward's units, of one query tile or two, the items and the joins: a block has between one item
    # and one for every four tiles, whatever the number of SMs that the host counts
    rest = got - fixed
    fwd = [up(16 * -(-n // (tt * k))) for k in (1, 2)]
    least, most = up(32 * len(tiles)), up(32 * sum(-(-t // 4) for t in tiles)) + up(16 * len(tiles))
    assert any(least <= rest - f <= most for f in fwd), (rest, fwd, least, most)


def test_refused(lib):
    for lengths, kw, text in [
        ([5, -1], {}, b"negative"), ([5, 6], dict(rows=10), b"more tokens"), ([5], dict(rows=0), b"positive"), ([5], dict(Hq=0), b"positive"),
        ([5], dict(Hkv=-2), b"positive"), ([5], dict(window=0), b"window"), ([5], dict(Hq=6, Hkv=4), b"Hq / Hkv"), ([5], dict(Hq=64, Hkv=2), b"Hq / Hkv"),
        ([5], dict(rows=2 ** 23 + 1), b"2^23"), ([5], dict(rows=2 ** 23, Hq=256, Hkv=16), b"2^31"), ([2 ** 31 - 1] * 3, dict(rows=2 ** 23), b"more tokens"),
    ]:
        a = dict(Hq=8, Hkv=2, rows=100, window=10)
        a.update(kw)
        assert table_bytes(lib, lengths, **a) == 0
        assert text in lib.msa_last_error(), (lengths, kw)
    shape = msa.PackedShape(100, 8, 2, 64, 10)
    assert lib.msa_packed_table_bytes(ctypes.byref(shape), (ctypes.c_int32 * 1)(5), 1) == 0 and b"head dim" in lib.msa_last_error()
    assert lib.msa_packed_table_bytes(None, (ctypes.c_int32 * 1)(5), 1) == 0
    assert table_bytes(lib, [], 8, 2, 1, 1) > 0  # no sequence at all
    assert table_bytes(lib, [0, 0], 8, 2, 1, 1) > 0


def test_plans_refused(lib):
    P = ctypes.c_void_p
    A, ODD, NULL = P(0x10000), P(0x10008), P(0)
    shape = ctypes.byref(msa.PackedShape(100, 8, 2, 128, 10))
    arr = (ctypes.c_int32 * 1)(90)
    c = msa.PackedCounts()
    assert lib.msa_packed_plan(shape, arr, 1, None, A, 1 << 20, NULL) == 1
    assert lib.msa_packed_plan(shape, arr, 1, ctypes.byref(c), NULL, 1 << 20, NULL) == 1
    assert lib.msa_packed_plan(shape, arr, 1, ctypes.byref(c), ODD, 1 << 20, NULL) == 1
    assert lib.msa_packed_plan(shape, arr, 1, ctypes.byref(c), A, 64, NULL) == 3
    good = dict(rows=100, tokens=90, Hq=8, Hkv=2, window=10, fwd_tiles=1, fwd_units=3, dq_units=3, chunk=4, items=1, slots=0, joins=0)
    make = lambda **kw: msa.PackedCounts(*{**good, **kw}.values())  # noqa: E731
    size = lib.msa_packed_workspace_size(ctypes.byref(make()), msa.OP_PACKED_FORWARD)
    back = lib.msa_packed_workspace_size(ctypes.byref(make()), msa.OP_PACKED_BACKWARD)
    assert 0 < size < back
    assert lib.msa_packed_workspace_size(ctypes.byref(make()), msa.OP_FORWARD) == 0
    assert lib.msa_packed_workspace_size(None, msa.OP_PACKED_FORWARD) == 0
    fwd = lambda p, *a, t=A, n=1 << 20, s=0.1, w=size: lib.msa_packed_forward(  # noqa: E731
        ctypes.byref(p), t, n, *(a or [A] * 3), s, A, A, A, w, NULL)
    for kw in (dict(rows=0), dict(tokens=101), dict(tokens=-1), dict(Hq=0), dict(Hkv=0), dict(window=0), dict(fwd_units=4), dict(fwd_tiles=3),
               dict(dq_units=2), dict(items=0), dict(slots=-1), dict(joins=1), dict(rows=2 ** 23 + 1)):
        assert fwd(make(**kw)) == 1, kw
        assert lib.msa_packed_workspace_size(ctypes.byref(make(**kw)), msa.OP_PACKED_BACKWARD) == 0, kw
    assert fwd(make(Hq=6)) in (1, 2)
    assert fwd(make(), t=NULL) == 1 and fwd(make(), t=ODD) == 1 and fwd(make(), n=100) == 1
    assert fwd(make(), s=0.0) == 1 and fwd(make(), s=float("nan")) == 1 and fwd(make(), w=size - 1) == 3
    assert fwd(make(), A, NULL, A) == 1 and fwd(make(), A, A, ODD) == 1
    for i in range(9):
        a = [A] * 9
        a[i] = NULL
        assert lib.msa_packed_backward(ctypes.byref(make()), A, 1 << 20, *a[:6], 0.1, *a[6:], A, back, NULL) == 1
    assert lib.msa_packed_backward(ctypes.byref(make()), A, 1 << 20, *[A] * 6, 0.1, *[A] * 3, A, back - 1, NULL) == 3


def test_binding_refuses():
    import torch

    with pytest.raises(msa.MSAError, match="lengths"):
        msa.msa_packed_plan([3, -1], 8, 2)
    with pytest.raises(msa.MSAError, match="rows"):
        msa.msa_packed_plan([3, 4], 8, 2, rows=6)
    with pytest.raises(msa.MSAError, match="CUDA device"):
        msa.msa_packed_plan([3, 4], 8, 2, device="cpu")
    with pytest.raises(TypeError, match="PackedPlan"):
        msa.msa_packed_forward(torch.zeros(4, 8, 128, dtype=torch.bfloat16), None, None, None, 0.1)
