"""The sparse backward called again and again on one input.

Two calls differ in the order in which the fp32 accumulators take the (token, key block) contributions, at
most top_k of a dQp row, each of which has the same bits in every call.
"""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300.inputs import Workload, make_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("return_kl, runs", [(True, 300), (False, 100)])
def test_proxy_gradients_of_repeated_calls(return_kl, runs):
    w = Workload("repeats", B=2, S=32768, Hq=16, Hkv=2, Hp=2, top_k=8)
    g = make_inputs(w, 43, device="cuda")
    shape = msa.make_shape(g["q"], g["k"], g["qp"], w.top_k, w.scale)
    o, lse, idx = msa.msa_forward(g["q"], g["k"], g["v"], g["qp"], g["kp"], w.top_k, w.scale)
    ws = msa.workspace(shape, msa.OP_BACKWARD, "cuda")

    def dqp():
        return msa.msa_backward(g["q"], g["k"], g["v"], g["qp"], g["kp"], o, lse, g["dout"], idx, w.top_k,
                                w.scale, ws=ws, return_kl=return_kl)[3].float()

    ref = dqp()
    # n <= 8 numbers summed in two orders differ by at most 2 (n - 1) 2^-24 sum |c|; with contributions up to
    # 32 times the row's largest element (they are of its size: the proxy keys of different blocks are independent) this is
    # 14 * 8 * 32 * 2^-24 < 2^-12 of it.  Rounding both to bf16 adds a step, 2^-7 of the element, where the two lie on
    # either side of a border.
    bound = 2.0 ** -7 * ref.abs() + 2.0 ** -12 * ref.abs().amax(-1, keepdim=True)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(runs):
        off += ((dqp() - ref).abs() > bound).sum()
    assert int(off) == 0, f"{int(off)} elements of dQp differ between calls"
    assert msa.msa_device_status(ws) == 0
