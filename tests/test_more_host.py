"""Refusals of the 4-bit cache, packed-prompt and several-axes entry points, all on the host before any launch."""
import ctypes

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build
from tests.test_local_host import A, NULL, P, part, rope_shape

ODD = P(0x10008)


@pytest.fixture(scope="module")
def lib():
    return msa.load_library(build.build())


def axes(count=3, of=(0, 1, 2)):
    return msa.RopeAxes(count, (ctypes.c_uint8 * 64)(*(of[i % len(of)] for i in range(64))))


def rope(lib, which, p=None, s=None, ax=None, pos=A, seq=A, ws=1 << 20):
    s, arr = ctypes.byref(s or rope_shape()), (msa.RopePart * 1)(p or part())
    ax = None if ax is None else ctypes.byref(ax)
    if which == "forward":
        return lib.msa_norm_rope_axes_forward(s, arr, 1, pos, A, ax, NULL)
    if which == "append":
        return lib.msa_norm_rope_axes_append(s, arr, 1, seq, pos, A, ax, A, ws, NULL)
    return lib.msa_norm_rope_axes_backward(s, arr, 1, pos, A, ax, A, ws, NULL)


@pytest.mark.parametrize("which", ["forward", "append", "backward"])
@pytest.mark.parametrize("kw,rc", [
    (dict(pos=NULL), 1), (dict(ax=axes(0, (0,))), 2), (dict(ax=axes(5)), 2), (dict(ax=axes(2)), 1), (dict(ax=axes(-1, (0,))), 2),
    (dict(pos=P(0x10002)), 1), (dict(ax=axes(), s=rope_shape(rotary=8)), 2),
])
def test_axes_refused(lib, which, kw, rc):
    assert rope(lib, which, **kw) == rc


def test_append_needs_lengths_and_a_workspace(lib):
    assert rope(lib, "append", ax=axes(), seq=NULL) == 1
    assert rope(lib, "append", ax=axes(), ws=8) == 3


@pytest.mark.parametrize("flags,cap,rc", [(8 | 2, 1024, 1), (8, 1000, 2), (16, 1024, 1)])
def test_cache_flags_refused(lib, flags, cap, rc):
    arr = (msa.RopePart * 1)(part(flags=flags))
    s = rope_shape(capacity=cap)
    assert lib.msa_norm_rope_append(ctypes.byref(s), arr, 1, A, A, A, 1 << 20, NULL) == rc


def test_cache_in_4_bits_only_in_an_append(lib):
    arr = (msa.RopePart * 1)(part(flags=8))
    assert lib.msa_norm_rope_forward(ctypes.byref(rope_shape(capacity=1024)), arr, 1, NULL, A, NULL) == 1


def test_caches_in_4_bits_that_overlap(lib):
    """Two parts with caches of 9344 bytes a head and block: side by side, and one byte row short of it."""
    s = rope_shape(B=1, N=1, capacity=128, rotary=0)
    n = lib.msa_q4_cache_bytes(1, 2, 128)
    assert n == 2 * 9344
    for off in (0, 16, n - 16):
        arr = (msa.RopePart * 2)(part(x=0x1000000, y=0x2000000, flags=8), part(x=0x1100000, y=0x2000000 + off, flags=8))
        assert lib.msa_norm_rope_append(ctypes.byref(s), arr, 2, A, NULL, A, 1 << 20, NULL) == 1
        assert b"same output" in lib.msa_last_error()
    # over its own input too
    arr = (msa.RopePart * 1)(part(x=0x2000000, y=0x2000000, flags=8))
    assert lib.msa_norm_rope_append(ctypes.byref(s), arr, 1, A, NULL, A, 1 << 20, NULL) == 1


@pytest.mark.parametrize("change,text", [
    (dict(B=0), b"positive"), (dict(window=0), b"window"), (dict(sinks=-1), b"sinks"), (dict(scale=0.0), b"scale"), (dict(D=64), b"head dim"),
    (dict(S=1000), b"multiple of 128"), (dict(Hq=6), b"Hq / Hkv"), (dict(Hq=64), b"Hq / Hkv"),
])
def test_window_decode_refused(lib, change, text):
    kw = dict(B=1, S=1024, Hq=8, Hkv=2, D=128, window=128, sinks=4, scale=0.1)
    kw.update(change)
    s = ctypes.byref(msa.WindowShape(*kw.values()))
    assert lib.msa_window_workspace_size(s, msa.OP_WINDOW_DECODE_Q4) == 0 and text in lib.msa_last_error()
    assert lib.msa_window_decode_q4(s, A, A, A, A, A, A, A, 1 << 40, NULL) in (1, 2) and text in lib.msa_last_error()


def test_decode_pointers_refused(lib):
    w = ctypes.byref(msa.WindowShape(1, 1024, 8, 2, 128, 128, 4, 0.1))
    m = ctypes.byref(msa.Shape(1, 1024, 8, 2, 2, 128, 4, 0.1))
    nw, nm = lib.msa_window_workspace_size(w, msa.OP_WINDOW_DECODE_Q4), lib.msa_workspace_size(m, msa.OP_DECODE_Q4)
    assert nw > 0 and nm > 0
    assert lib.msa_window_decode_q4(None, A, A, A, A, A, A, A, nw, NULL) == 1
    assert lib.msa_decode_q4(None, A, A, A, A, A, A, A, A, A, A, nm, NULL) == 1
    for bad in (NULL, ODD):
        for i in range(6):
            args = [A] * 6
            args[i] = bad
            if not (bad is ODD and i == 3):  # lengths are words
                assert lib.msa_window_decode_q4(w, *args, A, nw, NULL) == 1, i
        for i in range(9):
            args = [A] * 9
            args[i] = bad
            if not (bad is ODD and i == 5):
                assert lib.msa_decode_q4(m, *args, A, nm, NULL) == 1, i
    assert lib.msa_window_decode_q4(w, *[A] * 6, A, nw - 1, NULL) == 3
    assert lib.msa_decode_q4(m, *[A] * 9, A, nm - 1, NULL) == 3
    bad = ctypes.byref(msa.Shape(1, 1000, 8, 2, 2, 128, 4, 0.1))
    assert lib.msa_workspace_size(bad, msa.OP_DECODE_Q4) == 0
    assert lib.msa_decode_q4(bad, *[A] * 9, A, nm, NULL) == 2


def test_read_refused(lib):
    assert lib.msa_q4_cache_bytes(1, 1, 100) == 0 and lib.msa_q4_cache_bytes(0, 1, 128) == 0 and lib.msa_q4_cache_bytes(1, -1, 128) == 0
    for args in [(0, 1, 128, 0, 1), (1, 0, 128, 0, 1), (1, 1, 100, 0, 1), (1, 1, 128, -1, 1), (1, 1, 128, 0, 0), (1, 1, 128, 0, 129),
                 (1, 1, 128, 128, 1), (1, 1, 128, 1, 2 ** 31 - 1)]:
        assert lib.msa_q4_read(A, *args, A, NULL) == 1, args
    assert lib.msa_q4_read(NULL, 1, 1, 128, 0, 1, A, NULL) == 1
    assert lib.msa_q4_read(A, 1, 1, 128, 0, 1, ODD, NULL) == 1


def test_binding_refuses():
    with pytest.raises(msa.MSAError, match="multiple of 128"):
        msa.msa_q4_cache(1, 2, 1000, "cpu")
    c = msa.msa_q4_cache(1, 2, 256, "cpu")
    assert c.shape == (1, 2, 2, 9344) and c.dtype == torch.uint8
    with pytest.raises(msa.MSAError, match="CUDA"):
        msa.msa_q4_read(c, 0, 1)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(msa.MSAError, match="CUDA"):
        msa.msa_window_decode_q4(q, c, c, torch.ones(1, dtype=torch.int32), 8, 0, 0.1)
    with pytest.raises(msa.MSAError, match="axes"):
        msa._axes((0, 1, 4), 3)
    with pytest.raises(msa.MSAError, match="pairs"):
        msa._axes((0, 1), 3)
    with pytest.raises(msa.MSAError, match="axes"):
        msa._axes((0, -1, 1), 3)


@pytest.mark.parametrize("bad", [[-1], (5, -2 ** 31), [2 ** 31], [2 ** 40, 1], [-2 ** 40], [1.0, -3.0], torch.tensor([4, -1])])
def test_lengths_out_of_range(bad):
    with pytest.raises(msa.MSAError, match="lengths must be in"):
        msa.msa_packed_plan(bad, 2, 1, device="cuda:0")


@pytest.mark.parametrize("bad", [[2.5], [2.7, 3.9], (4, 0.5), [float("nan")], [1, float("inf")], ["3"], [None], [[1, 2]],
                                 torch.tensor([1.0, 2.5]), torch.tensor([[1, 2]])])
def test_lengths_that_are_no_whole_numbers(bad):
    with pytest.raises(msa.MSAError, match="lengths must be whole numbers"):
        msa.msa_packed_plan(bad, 2, 1, device="cuda:0")


@pytest.mark.parametrize("kw", [dict(heads=2.5), dict(kv_heads=0.5), dict(rows=9.5), dict(rows=float("nan"))])
def test_sizes_that_are_no_whole_numbers(kw):
    with pytest.raises(msa.MSAError, match=f"{list(kw)[0]} must be whole numbers"):
        msa.msa_packed_plan(**{"lengths": [4, 5], "heads": 2, "kv_heads": 1, "device": "cuda:0", **kw})
