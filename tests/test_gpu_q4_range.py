"""Decode over caches in 4 bits where the sizes of rows lie far apart: exponents of V that move the running maximum by more
than 2^126."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
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
