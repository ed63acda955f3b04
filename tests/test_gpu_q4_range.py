"""Decode over caches in 4 bits where the sizes of rows lie far apart: exponents of V that move the running maximum by more
than 2^126, rows that no call has written, weights far below the largest,
elements of q far below their head's largest."""
import math

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_q4 as plain
from tests.plain_local import F, HALF, check
from tests.test_gpu_q4 import SCALE, decode_check, gen, lens32

pytestmark = pytest.mark.gpu


def caches(k, v, cap):
    B, n, H = k.shape[:3]
    out = [msa.msa_q4_cache(B, H, cap, "cuda") for _ in range(2)]
    for c, x in zip(out, (k, v)):
        msa.msa_norm_rope_append([x], None, None, lens32(*[n] * B), [c])
    return out


@pytest.mark.parametrize("power", [20, 37, 60, 90])
@pytest.mark.parametrize("n, zeros", [(256, slice(0, 128)), (128, slice(0, 32)), (128, slice(96, 128)), (8192, slice(0, 4000)),
                                      (8192, slice(64, 8190))])
def test_zero_values_beside_large_ones(n, zeros, power):
    """Zero rows (of the least exponent) in front of large ones in one warp's keys, in another warp's, and in other
    parts of the sequence.  Keys of zero values count in the softmax like any other."""
    r = gen(n + power)
    k, v = r(1, n, 2, 128, scale=0.5), r(1, n, 2, 128) * 2.0 ** power
    v[:, zeros] = 0
    kc, vc = caches(k, v, n)
    q = r(1, 16, 128)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(n), n, 0, SCALE)
    decode_check(q, kc, vc, [n], lambda b, m: torch.arange(m, device="cuda"), o, lse, n)


@pytest.mark.parametrize("B, H, Hq, n", [(1, 1, 1, 300), (1, 2, 8, 5000), (64, 8, 64, 2048), (40, 8, 128, 3000)])
@pytest.mark.parametrize("written", [0, 1, 700])
def test_rows_never_written(B, H, Hq, n, written):
    """A new cache holds zeros, and its rows stand for rows of zeros: they weigh 1 each (their scores are 0)."""
    r = gen(B + n)
    cap = (n + 127) // 128 * 128
    kc, vc = (msa.msa_q4_cache(B, H, cap, "cuda") for _ in range(2))
    w = min(written, n)
    if w:  # the last ones, as a decoding program writes them
        for c in (kc, vc):
            msa.msa_norm_rope_append([r(B, w, H, 128, scale=0.5)], None, None, lens32(*[n] * B), [c])
    q = r(B, Hq, 128)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(*[n] * B), n, 0, SCALE)
    if w == 0:
        assert (o == 0).all()
        assert (lse - math.log(n)).abs().max() <= F
        return
    k, v = (plain.values(plain.unpack(c[[0, -1]])) for c in (kc, vc))
    for i, b in ((0, 0), (1, B - 1)):
        want = plain.attend(q[b], k[i, :n], v[i, :n], SCALE)
        check(f"o[{b}]", o[b], want["o"])
        check(f"lse[{b}]", lse[b], want["lse"])


def test_sparse_rows_never_written():
    B, cap = 2, 2048
    kc, vc = (msa.msa_q4_cache(B, 8, cap, "cuda") for _ in range(2))
    r = gen(3)
    q, qp, kp = r(B, 64, 128), r(B, 8, 128), r(B, cap, 1, 128)
    o, lse, idx = msa.msa_decode_q4(q, qp, kc, vc, kp, lens32(2048, 1500), 12, SCALE)
    assert (o == 0).all()
    assert (idx[1] == torch.arange(12, device="cuda", dtype=torch.int32)).all()  # all of the shorter sequence's blocks
    for b, keys in ((0, 12 * 128), (1, 1500)):
        assert (lse[b] - math.log(keys)).abs().max() <= F


@pytest.mark.parametrize("B, H, Hq, n", [(57, 8, 8, 16384), (38, 8, 128, 16384)])
def test_one_heavy_key_among_many_light_ones(B, H, Hq, n):
    """A first token 2^26 times as heavy as any of the 16383 others, whose values alone reach the upper 64 dims: their weights are
    far below fp16's normal range.  Relative to a warp's largest weight they are off by at most 2^-31 (half a step of 2^-24 where the largest is
    at least 2^6)."""
    q = torch.full((B, Hq, 128), 1.0625, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, n, H, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[:, 0] = 1.5
    v[:, 0, :, 64:] = 0
    kc, vc = caches(k.expand(B, n, H, 128), v.expand(B, n, H, 128), n)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(*[n] * B), n, 0, SCALE)
    for b in (0, B - 1):
        kb, vb = (plain.values(plain.unpack(c[b:b + 1]))[0] for c in (kc, vc))
        want = plain.attend(q[b], kb, vb, SCALE)
        ref = want["o"][0]
        # (a row's largest kept value is between 1536 and half of that times its power of two: the factor 2)
        bound = HALF * ref.abs() + (plain.HALF16 + F) * ref.abs() + n * 2.0 ** -31 * 2
        check(f"o[{b}]", o[b], (ref, bound))
        check(f"lse[{b}]", lse[b], want["lse"])


def test_small_elements_of_q():
    """All but one element of every head 2^-20 of the largest, whose keys are 0 there: the scores are theirs alone."""
    r = gen(11)
    n, H, Hq = 600, 2, 32
    q = r(1, Hq, 128) * 2.0 ** -20
    q[..., 5] = 1.0
    k = r(1, n, H, 128) * 2.0 ** 20
    k[..., 5] = 0
    kc, vc = caches(k, r(1, n, H, 128), 640)
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(n), n, 0, SCALE)
    decode_check(q, kc, vc, [n], lambda b, m: torch.arange(m, device="cuda"), o, lse, 640)


def test_a_head_of_infinities_or_of_the_smallest_numbers():
    """q's power of two at its ends: a head of bf16's subnormal numbers scores 0, one with an infinity is NaN, one of
    the largest numbers is what its scores make of it, and no head reaches another."""
    r = gen(12)
    kc, vc = caches(r(1, 200, 1, 128, scale=2.0 ** -100), r(1, 200, 1, 128), 256)
    q = r(1, 8, 128)
    q[0, 0] = 2.0 ** -133
    q[0, 1] = 0
    q[0, 2] = q[0, 2].abs().clamp(min=0.5) * 2.0 ** 97
    q[0, 3, 7] = float("inf")
    q[0, 4, 7] = float("nan")
    q[0, 5] *= 2.0 ** 100
    o, lse = msa.msa_window_decode_q4(q, kc, vc, lens32(200), 200, 0, SCALE)
    fine = [0, 1, 2, 5, 6, 7]
    assert torch.isnan(lse[0, [3, 4]]).all() and torch.isnan(o[0, [3, 4]]).any(-1).all()
    decode_check(q[:, fine], kc, vc, [200], lambda b, m: torch.arange(m, device="cuda"), o[:, fine], lse[:, fine], 256)
