"""The operators together, as a serving program uses them: packed prompts of text and image tokens, normed and rotated by
positions of several axes, attended packed, their keys and values stored in 4 bits, and tokens decoded on these caches."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local, plain_q4
from tests.plain_local import check
from tests.test_gpu_axes import plain_axes

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def test_prompts_then_tokens():
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    Hq, H, cap = 8, 2, 512
    lengths = [300, 37, 128]
    rows, heads, B = sum(lengths), [Hq, H, H], len(lengths)
    w = [1 + 0.1 * torch.randn(128, generator=g, device="cuda") for _ in range(2)]
    how = dict(rotate=[True, True, False], axes=[0] * 16 + [1] * 24 + [2] * 24)
    freq = 10000.0 ** (-torch.arange(0, 128, 2, device="cuda") / 128)
    x = torch.randn((1, rows, sum(heads), 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.cat([torch.stack([t // 20, t // 5 % 4, t % 5]) for t in (torch.arange(n, device="cuda") for n in lengths)], 1)
    q, k, v = msa.msa_norm_rope_forward(x.split(heads, 2), [*w, None], freq, positions=pos[:, None].int().contiguous(), **how)
    for got, part, wi in zip((q, k), x.split(heads, 2), w):
        check("rotated", got, plain_axes(part, wi, pos[:, None], freq, how["axes"], False)["y"])

    plan = msa.msa_packed_plan(lengths, Hq, H, device="cuda")
    o, lse = msa.msa_packed_forward(q[0], k[0], v[0], plan, SCALE)
    caches = [msa.msa_q4_cache(B, H, cap, "cuda") for _ in range(2)]
    kp = torch.randn((B, cap, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    at = 0
    for b, n in enumerate(lengths):
        s = slice(at, at + n)
        at += n
        want = plain_local.window(q[:, s], k[:, s], v[:, s], n, 0, SCALE)
        check("o", o[None, s], want["o"])
        check("lse", lse[None, :, s], want["lse"])
        msa.msa_norm_rope_append([k[:, s], v[:, s]], None, None, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                 [c[b:b + 1] for c in caches])
        for c, t in zip(caches, (k, v)):
            assert torch.equal(msa.msa_q4_read(c, 0, n)[b].double(), plain_q4.values(plain_q4.quantise(t[0, s])))

    seq_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for step in range(3):
        seq_len += 1
        x = torch.randn((B, 1, sum(heads), 128), generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.full((3, B, 1), 1000 + step, dtype=torch.int32, device="cuda")
        yq, _, _ = msa.msa_norm_rope_append(x.split(heads, 2), [*w, None], freq, seq_len, [None, *caches], positions=pos, **how)
        qn = yq[:, 0].contiguous()
        o, lse = msa.msa_window_decode_q4(qn, *caches, seq_len, 200, 4, SCALE)
        qp = torch.randn((B, H, 128), generator=g, device="cuda").to(torch.bfloat16)
        so, slse, idx = msa.msa_decode_q4(qn, qp, *caches, kp, seq_len, 2, SCALE)
        kv = [plain_q4.values(plain_q4.unpack(c)) for c in caches]
        for b, n in enumerate(seq_len.tolist()):
            j = plain_q4.window_keys(n, 200, 4, "cuda")
            want = plain_q4.attend(qn[b], kv[0][b, j], kv[1][b, j], SCALE)
            check("window", o[b], want["o"])
            check("window lse", lse[b], want["lse"])
            for h in range(H):
                j = torch.cat([torch.arange(128 * i, min(n, 128 * i + 128), device="cuda") for i in idx[b, h].tolist() if i >= 0])
                hs = slice(4 * h, 4 * h + 4)
                want = plain_q4.attend(qn[b, hs], kv[0][b, j][:, h:h + 1], kv[1][b, j][:, h:h + 1], SCALE)
                check("sparse", so[b, hs], want["o"])
                check("sparse lse", slse[b, hs], want["lse"])
