"""Refusals of the window and norm-and-rotation entry points, all on the host before any launch, and the host
rules that size their work."""
import ctypes

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build

P = ctypes.c_void_p
A = P(0x10000)  # aligned, never dereferenced: every call here fails on the host
NULL = P(0)


@pytest.fixture(scope="module")
def lib():
    return msa.load_library(build.build())


def shape(B=1, S=1000, Hq=8, Hkv=2, D=128, window=128, sinks=4, scale=0.1):
    return msa.WindowShape(B, S, Hq, Hkv, D, window, sinks, scale)


@pytest.mark.parametrize("change,text", [
    (dict(B=0), b"positive"), (dict(S=0), b"positive"), (dict(Hq=-8), b"positive"), (dict(Hkv=0), b"positive"),
    (dict(window=0), b"window"), (dict(sinks=-1), b"sinks"), (dict(scale=0.0), b"scale"),
    (dict(scale=float("nan")), b"scale"), (dict(scale=float("inf")), b"scale"), (dict(D=64), b"head dim"),
    (dict(S=2 ** 23 + 1), b"2^23"), (dict(Hq=6), b"Hq / Hkv"), (dict(Hq=9), b"Hq / Hkv"),
    (dict(Hq=64, Hkv=2), b"Hq / Hkv"), (dict(B=2 ** 15, S=2 ** 16), b"2^31"), (dict(S=2 ** 23, Hq=512, Hkv=64), b"2^32"),
])
def test_window_shapes_refused(lib, change, text):
    s = shape(**change)
    for op in (msa.OP_WINDOW_FORWARD, msa.OP_WINDOW_BACKWARD):
        assert lib.msa_window_workspace_size(ctypes.byref(s), op) == 0
        assert text in lib.msa_last_error()
    assert lib.msa_window_forward(ctypes.byref(s), A, A, A, A, A, A, 1 << 40, NULL) in (1, 2)
    assert text in lib.msa_last_error()


def test_window_arguments_refused(lib):
    s = ctypes.byref(shape())
    odd = P(0x10008)
    size = lib.msa_window_workspace_size(s, msa.OP_WINDOW_FORWARD)
    assert size > 0
    assert lib.msa_window_workspace_size(s, msa.OP_DECODE) == 0
    assert lib.msa_window_forward(None, A, A, A, A, A, A, size, NULL) == 1
    for i in range(5):
        args = [A] * 5
        args[i] = NULL
        assert lib.msa_window_forward(s, *args, A, size, NULL) == 1
        args[i] = odd
        assert lib.msa_window_forward(s, *args, A, size, NULL) == 1 and b"aligned" in lib.msa_last_error()
    assert lib.msa_window_forward(s, A, A, A, A, A, NULL, size, NULL) == 1
    assert lib.msa_window_forward(s, A, A, A, A, A, A, size - 1, NULL) == 3
    for i in range(9):
        args = [A] * 9
        args[i] = NULL
        assert lib.msa_window_backward(s, *args, A, 1 << 40, NULL) == 1
    assert lib.msa_window_backward(s, *[A] * 9, A, size, NULL) == 3
    for i in range(6):
        args = [A] * 6
        args[i] = NULL
        assert lib.msa_window_decode(s, *args, A, 1 << 40, NULL) == 1
    assert lib.msa_window_decode(s, *[A] * 6, A, 0, NULL) == 3


def test_window_workspace_stays_small(lib):
    """The backward keeps eight bytes per query row and a bounded number of key-block partials."""
    for B, S, Hq, Hkv, W, ns in ((1, 65536, 64, 8, 512, 4), (1, 1 << 20, 16, 4, 4096, 130), (1, 32768, 32, 8, 32768, 0),
                                 (1, 65536, 64, 64, 1, 4), (1, 1 << 20, 4, 4, 100, 4000)):
        s = shape(B, S, Hq, Hkv, window=W, sinks=ns)
        size = msa.msa_window_workspace_size(s, msa.OP_WINDOW_BACKWARD)
        blocks = B * Hkv * -(-S // 128)
        assert size <= B * S * Hq * 8 + (2 * 8 * 160 + 2 * blocks) * 2 * 128 * 128 * 4, (S, size)


def test_window_binding_refusals():
    q, k = torch.zeros(1, 8, 4, 128, dtype=torch.bfloat16), torch.zeros(1, 8, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(msa.MSAError, match="CUDA tensor"):
        msa.msa_window_forward(q, k, k, 4, 0, 0.1)
    with pytest.raises(msa.MSAError, match="4 dimensions"):
        msa.msa_window_forward(q[0], k, k, 4, 0, 0.1)
    with pytest.raises(TypeError):
        msa.msa_window_forward(None, k, k, 4, 0, 0.1)
    with pytest.raises(msa.MSAError, match="3 dimensions"):
        msa.msa_window_decode(q, k, k, torch.ones(1, dtype=torch.int32), 4, 0, 0.1)
    s = msa.make_window_shape(q, k, 2 ** 40, 2 ** 33, 0.1)  # larger than int32: everything
    assert s.window == s.sinks == 2 ** 31 - 1
    with pytest.raises(msa.MSAError, match="out of range"):
        msa.make_window_shape(q, k, -2 ** 40, 0, 0.1)


# ------------------------------------------------------------------------------------ norm, rotation
def part(**kw):
    p = msa.RopePart(x=0x10000, x_batch=1024, x_token=256, y=0x20000, y_batch=1024, y_token=256, dx=0x30000,
                     dx_batch=1024, dx_token=256, weight=0x40000, dweight=0x50000, heads=2, flags=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def rope_shape(**kw):
    s = msa.RopeShape(B=1, N=4, D=128, rotary=64, interleaved=0, capacity=16, eps=1e-6)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def calls(lib, s, p, n=1, pos=A, freq=A, ws=A, size=1 << 40):
    parts = (msa.RopePart * 9)(*[p] * 9)
    s = ctypes.byref(s)
    return (lib.msa_norm_rope_forward(s, parts, n, pos, freq, NULL),
            lib.msa_norm_rope_append(s, parts, n, pos, freq, ws, size, NULL),
            lib.msa_norm_rope_backward(s, parts, n, pos, freq, ws, size, NULL))


@pytest.mark.parametrize("kw,rc", [
    (dict(s=rope_shape(B=0)), 1), (dict(s=rope_shape(N=0)), 1), (dict(s=rope_shape(D=64)), 2),
    (dict(s=rope_shape(eps=-1.0)), 1), (dict(s=rope_shape(eps=float("nan"))), 1), (dict(s=rope_shape(eps=float("inf"))), 1),
    (dict(s=rope_shape(rotary=8)), 2), (dict(s=rope_shape(rotary=144)), 2), (dict(s=rope_shape(rotary=-16)), 2),
    (dict(s=rope_shape(B=2 ** 16, N=2 ** 15)), 2), (dict(n=0), 1), (dict(n=9), 2), (dict(freq=NULL), 1),
    (dict(pos=P(0x10002)), 1), (dict(p=part(x=0)), 1), (dict(p=part(y=0x20004)), 1), (dict(p=part(weight=0x40008)), 1),
    (dict(p=part(heads=0)), 2), (dict(p=part(heads=1025)), 2), (dict(p=part(flags=4)), 1), (dict(p=part(x_token=129)), 1),
    (dict(p=part(y_batch=4)), 1),
])
def test_rope_refused(lib, kw, rc):
    kw.setdefault("s", rope_shape())
    kw.setdefault("p", part())
    assert calls(lib, **kw) == (rc, rc, rc)


def test_rope_refused_by_one(lib):
    cache = part(flags=3)
    parts = (msa.RopePart * 1)(cache)
    s = rope_shape()
    assert lib.msa_norm_rope_forward(ctypes.byref(s), parts, 1, A, A, NULL) == 1
    assert b"MSA_ROPE_CACHE" in lib.msa_last_error()
    parts = (msa.RopePart * 1)(part(dx=0))
    assert lib.msa_norm_rope_backward(ctypes.byref(s), parts, 1, A, A, A, 1 << 40, NULL) == 1
    parts = (msa.RopePart * 1)(part(weight=0))
    assert lib.msa_norm_rope_backward(ctypes.byref(s), parts, 1, A, A, A, 1 << 40, NULL) == 1
    assert b"without a weight" in lib.msa_last_error()
    parts = (msa.RopePart * 1)(part())
    need = lib.msa_norm_rope_workspace_size(1, msa.OP_NORM_ROPE_BACKWARD)
    assert need > 256
    assert lib.msa_norm_rope_backward(ctypes.byref(s), parts, 1, A, A, A, need - 1, NULL) == 3
    assert lib.msa_norm_rope_append(ctypes.byref(s), parts, 1, A, A, A, 255, NULL) == 3
    assert lib.msa_norm_rope_append(ctypes.byref(s), parts, 1, NULL, A, A, 256, NULL) == 1  # no lengths
    small = rope_shape(capacity=3)
    assert lib.msa_norm_rope_append(ctypes.byref(small), parts, 1, A, A, A, 256, NULL) == 1
    assert lib.msa_norm_rope_workspace_size(0, msa.OP_NORM_ROPE_APPEND) == 0
    assert lib.msa_norm_rope_workspace_size(9, msa.OP_NORM_ROPE_APPEND) == 0
    assert lib.msa_norm_rope_workspace_size(1, msa.OP_DECODE) == 0


def test_rope_strides():
    """_rows on tensors that say they are on a GPU (nothing is launched)."""
    class Fake(torch.Tensor):
        is_cuda = True

    def fake(t):
        return t.as_subclass(Fake)

    base = fake(torch.zeros(4, 6, 10, 128, dtype=torch.bfloat16))
    assert msa._rows(base, "x")[1:] == (6 * 1280, 1280)
    assert msa._rows(base[:, ::2, 2:5], "x", 4, 3, 3)[1:] == (6 * 1280, 2560)
    assert msa._rows(base[:1], "x")[1] == 0  # one sequence: no batch stride
    assert msa._rows(base.transpose(0, 1), "x", write=True)[1:] == (1280, 7680)
    for bad in (base.transpose(2, 3), base[..., ::2], base[:, :, ::2], base[0], base[..., :64],
                fake(torch.zeros(1, 2, 3, 128))):
        with pytest.raises(msa.MSAError):
            msa._rows(bad, "x")
    with pytest.raises(msa.MSAError, match="aligned"):
        msa._rows(fake(torch.zeros(4 * 129 * 2, dtype=torch.bfloat16).as_strided((2, 2, 1, 128), (258, 129, 128, 1))), "x")
    wide = fake(torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)).expand(1, 5, 2, 128)
    assert msa._rows(wide, "x")[2] == 0  # read five times
    with pytest.raises(msa.MSAError, match="overlaps"):
        msa._rows(wide, "dx", write=True)
    with pytest.raises(msa.MSAError, match="overlaps"):
        msa._rows(fake(torch.zeros(4096, dtype=torch.bfloat16)).as_strided((2, 5, 2, 128), (256, 256, 128, 1)), "dx", write=True)
    with pytest.raises(msa.MSAError, match="expected"):
        msa._rows(base, "x", 4, 6, 9)


def test_rope_binding_refusals():
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(msa.MSAError, match="CUDA tensor"):
        msa.msa_norm_rope_forward([x], [None], None)
    with pytest.raises(TypeError):
        msa.msa_norm_rope_forward([], [], None)
    with pytest.raises(TypeError):
        msa.msa_norm_rope_append([None], [None], None, x, [None])


def test_rope_outputs_are_distinct(lib):
    """One cache (or gradient) given for two parts would be written by both."""
    s = ctypes.byref(rope_shape())
    two = lambda **kw: (msa.RopePart * 2)(part(), part(**kw))  # noqa: E731
    a = part()
    other = dict(y=a.y + 4096, dx=a.dx + 4096, dweight=a.dweight + 4096)
    for clash in ("y", "dx", "dweight"):
        parts = two(**{k: v for k, v in other.items() if k != clash})
        if clash == "y":  # backward only reads it
            assert lib.msa_norm_rope_forward(s, parts, 2, A, A, NULL) == 1
            assert b"same output" in lib.msa_last_error()
            assert lib.msa_norm_rope_append(s, parts, 2, A, A, A, 1 << 40, NULL) == 1
        else:
            assert lib.msa_norm_rope_backward(s, parts, 2, A, A, A, 1 << 40, NULL) == 1
        assert b"same output" in lib.msa_last_error()
