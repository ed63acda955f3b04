"""Lengths, positions and frequencies that start anywhere in a larger tensor."""
import ctypes

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build

P = ctypes.c_void_p
A, NULL = P(0x10000), P(0)
DEV = "cuda:0"


@pytest.mark.parametrize("at", [0x20004, 0x20008, 0x2000c, 0x20002, 0x20001])
def test_alignment_of_words(at):
    """Four bytes are enough for what is read four bytes at a time; the calls end at their workspace of no bytes."""
    lib = msa.load_library(build.build())
    s = msa.RopeShape(1, 4, 128, 64, 0, 16, 1e-6)
    part = (msa.RopePart * 1)(msa.RopePart(0x30000, 0, 256, 0x40000, 0, 256, 0x50000, 0, 256, 0, 0, 2, 1))
    word = P(at)
    want = 3 if at % 4 == 0 else 1
    r = ctypes.byref(s)
    assert lib.msa_norm_rope_append(r, part, 1, word, A, A, 0, NULL) == want
    assert lib.msa_norm_rope_append(r, part, 1, A, word, A, 0, NULL) == want
    assert lib.msa_norm_rope_backward(r, part, 1, word, A, A, 0, NULL) == want
    assert lib.msa_norm_rope_backward(r, part, 1, A, word, A, 0, NULL) == want
    w = msa.WindowShape(1, 1000, 8, 2, 128, 100, 4, 0.1)
    assert lib.msa_window_decode(ctypes.byref(w), A, A, A, word, A, A, A, 0, NULL) == want
    d = msa.Shape(1, 1024, 8, 2, 2, 128, 4, 0.1)
    assert lib.msa_decode(ctypes.byref(d), A, A, A, A, A, word, A, A, A, A, 0, NULL) == want
    assert (b"4-byte" in lib.msa_last_error()) == (want == 1)
    # no lengths at all
    assert lib.msa_window_decode(ctypes.byref(w), A, A, A, NULL, A, A, A, 0, NULL) == 1
    assert lib.msa_decode(ctypes.byref(d), A, A, A, A, A, NULL, A, A, A, A, 0, NULL) == 1


def rnd(*shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.gpu
def test_norm_rope_of_slices():
    x, dy = rnd(3, 7, 4, 128, seed=1), rnd(3, 7, 4, 128, seed=2)
    w = torch.linspace(0.5, 1.5, 128, device=DEV)
    freqs = 10000.0 ** (-torch.arange(0, 65, 2, device=DEV) / 64)
    pos = torch.arange(21, dtype=torch.int32, device=DEV).view(3, 7) * 1001
    f = freqs[1:]
    args = dict(positions=pos[1:], interleaved=True)  # 28 bytes into pos, 4 into freqs
    assert args["positions"].data_ptr() % 16 and f.data_ptr() % 16
    y, = msa.msa_norm_rope_forward([x[1:]], [w], f, **args)
    (dx,), (dw,) = msa.msa_norm_rope_backward([x[1:]], [w], [dy[1:]], f, **args)
    args["positions"] = pos[1:].clone()
    y2, = msa.msa_norm_rope_forward([x[1:]], [w], f.clone(), **args)
    (dx2,), (dw2,) = msa.msa_norm_rope_backward([x[1:]], [w], [dy[1:]], f.clone(), **args)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_serving_the_rest_of_a_batch():
    """Append, window step and sparse step of sequences 1 .. B - 1, with slices of the batch's tensors."""
    B, cap, scale = 4, 256, 128 ** -0.5
    lens = torch.tensor([9, 200, 256, 31], dtype=torch.int32, device=DEV)
    x = rnd(B, 13, 128, seed=3)
    kc, vc, pc = rnd(B, cap, 2, 128, seed=4), rnd(B, cap, 2, 128, seed=5), rnd(B, cap, 1, 128, seed=6)
    f = 10000.0 ** (-torch.arange(0, 64, 2, device=DEV) / 64)

    def step(n, x, kc, vc, pc):
        q, _, _, qp, _ = msa.msa_norm_rope_append(list(x.split((6, 2, 2, 2, 1), 1)), None, f, n, [None, kc, vc, None, pc])
        q = torch.cat([q, q[:, :2]], 1)  # eight heads
        return (q, qp) + msa.msa_window_decode(q, kc, vc, n, 50, 4, scale) + \
            msa.msa_decode(q, qp, kc, vc, pc, n, 2, scale)

    whole = [t.clone() for t in (kc, vc, pc)]
    want = step(lens, x, *whole)
    got = step(lens[1:], x[1:], kc[1:], vc[1:], pc[1:])
    assert lens[1:].data_ptr() % 16
    assert all(torch.equal(a[1:], b) for a, b in zip(want, got))
    assert all(torch.equal(a[1:], b[1:]) for a, b in zip(whole, (kc, vc, pc)))
