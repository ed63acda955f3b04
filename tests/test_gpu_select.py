"""The decode step's selection: rows of some blocks have a kernel of their own, which picks what the other one picks."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
MANY = 1025 * 128  # a capacity at which every row is merged from sorted lists


def select(qp, kp, n, top_k, cap):
    B, Hp = qp.shape[:2]
    pad = torch.zeros((B, cap - kp.shape[1], 1, 128), dtype=torch.bfloat16, device="cuda")
    kp = torch.cat([kp, pad], 1)
    kv = torch.zeros((B, cap, 1, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((B, max(4, Hp), 128), dtype=torch.bfloat16, device="cuda")
    return msa.msa_decode(q, qp, kv, kv, kp.contiguous(), n, top_k, SCALE)[2]


def plain(qp, kp, n, top_k):
    """Blocks by score, ties to the lower one, a sorted list each: quarters, so every order of summation is exact."""
    out = []
    for b, m in enumerate(n.tolist()):
        last = (m - 1) // 128
        z = (qp[b].double() @ kp[b, :, 0].double().T).view(qp.shape[1], -1, 128).amax(-1)
        for p in range(qp.shape[1]):
            best = sorted(range(last), key=lambda i: (-float(z[p, i]), i))[:top_k - 1]
            row = sorted(best) + [last]
            out.append(row + [-1] * (top_k - len(row)))
    return torch.tensor(out, dtype=torch.int32).view(len(n), qp.shape[1], top_k)


@pytest.mark.parametrize("blocks,top_k,Hp", [(1, 1, 1), (2, 2, 2), (33, 5, 4), (64, 16, 2), (64, 64, 1), (65, 16, 4), (200, 33, 2), (256, 7, 1), (257, 16, 2), (1024, 64, 1)])
@pytest.mark.parametrize("coarse", [False, True])
def test_few_blocks_as_many(blocks, top_k, Hp, coarse):
    g = torch.Generator(device="cuda")
    g.manual_seed(blocks + top_k)
    B, cap = 3, 128 * blocks
    quarter = lambda *s: (torch.randn(s, generator=g, device="cuda") * 4).round() / 4  # noqa: E731
    qp, kp = quarter(B, Hp, 128), quarter(B, cap, 1, 128)
    if coarse:  # few different scores: ties in every row, among them +0 and -0
        qp[:] = 0
        qp[..., 0] = -0.25
        kp = kp.round().clamp(-1, 0)
    qp, kp = qp.to(torch.bfloat16), kp.to(torch.bfloat16)
    n = torch.tensor([cap, max(1, cap - 127), max(1, cap // 2)], dtype=torch.int32, device="cuda")
    got = select(qp, kp, n, top_k, cap)
    assert torch.equal(got.cpu(), plain(qp, kp, n, top_k))
    assert torch.equal(got, select(qp, kp, n, top_k, MANY))  # the kernel for more blocks


def test_scores_that_are_not_finite():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kp = torch.randn((1, 128 * 9, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    qp = torch.randn((1, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    n = torch.tensor([128 * 9], dtype=torch.int32, device="cuda")
    kp[0, 256:384] = float("nan")  # a whole block
    kp[0, 700, 0, 3] = float("inf")
    for top_k in (2, 4, 8, 9, 12):
        got = select(qp, kp, n, top_k, 128 * 9)
        assert torch.equal(got, select(qp, kp, n, top_k, MANY))
        assert not (got == 2).any()  # seven blocks have a score
    nan = torch.full_like(qp, float("nan"))
    assert torch.equal(select(nan, kp, n, 4, 128 * 9), select(nan, kp, n, 4, MANY))
    assert (select(nan, kp, n, 4, 128 * 9)[..., 0] == 8).all()  # the local block alone


@pytest.mark.parametrize("B,blocks,Hp", [(24, 300, 2), (64, 96, 1), (130, 47, 4), (2, 6000, 1)])
def test_large_capacities_of_many_sequences(B, blocks, Hp):
    """More blocks of capacity than CTAs: each takes several, of sequences of every length (the last a whole number of
    rounds, one block less and one more among them)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    cap, top_k = 128 * blocks, 9
    quarter = lambda *s: (torch.randn(s, generator=g, device="cuda") * 4).round() / 4  # noqa: E731
    qp, kp = quarter(B, Hp, 128).to(torch.bfloat16), quarter(B, cap, 1, 128).to(torch.bfloat16)
    n = torch.randint(1, cap + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0], n[1] = cap, 1
    for i, m in enumerate((128, 129, 256, 257, cap - 128, cap - 127, cap // 2, 5, 0, cap + 1)):
        if 2 + i < B:
            n[2 + i] = m
    kp[:, -1] = 100  # no score of the last block's keys reaches those of the others
    ok = [b for b, m in enumerate(n.tolist()) if 1 <= m <= cap]
    got = select(qp, kp, n, top_k, cap)[ok]
    assert torch.equal(got.cpu(), plain(qp[ok], kp[ok], n[ok], top_k))


@pytest.mark.parametrize("cap", [128 * 40, 128 * 300, MANY])
@pytest.mark.parametrize("top_k", [5, 16, 40])
def test_blocks_without_a_score_are_padding(cap, top_k):
    """Blocks of NaN are not picked, and the places that they leave are padded like any other: a row is ascending, ends with the
    local block, and holds -1 behind it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(top_k)
    kp = torch.randn((3, 128 * 40, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    qp = torch.randn((3, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    kp[1, :128 * 30] = float("nan")
    qp[2] = float("nan")
    n = torch.tensor([128 * 40, 128 * 39 + 5, 128 * 40], dtype=torch.int32, device="cuda")
    for b, (row, scored) in enumerate(zip(select(qp, kp, n, top_k, cap).tolist(), (39, 9, 0))):
        for ids in row:
            count = min(top_k - 1, scored) + 1
            assert ids[count - 1] == 39 and ids[count:] == [-1] * (top_k - count)
            assert ids[:count] == sorted(set(ids[:count])) and ids[0] >= (30 if b == 1 else 0)


@pytest.mark.parametrize("at", [0, 199])
def test_a_call_writes_its_own_status(at):
    """A length out of range is flagged wherever it stands, and the next call on the same workspace starts clear."""
    B, cap = 200, 256
    qp = torch.zeros((B, 1, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((B, cap, 1, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((B, 4, 128), dtype=torch.bfloat16, device="cuda")
    n = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    ws = torch.full((1 << 22,), 0xff, dtype=torch.uint8, device="cuda")
    for length, flagged in ((cap, False), (cap + 1, True), (0, True), (1, False)):
        n[at] = length
        msa.msa_decode(q, qp, kv, kv, kv, n, 2, SCALE, ws=ws)
        assert (msa.msa_device_status(ws) != 0) == flagged


def test_replays_of_a_captured_step_read_their_own_scores():
    """Selection and attention start while the kernel in front ends: with other queries, keys and lengths in the same
    memory every replay equals the eager step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    B, Hq, H, cap, top_k = 8, 32, 4, 128 * 40, 8
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, qp, kp = rand(B, Hq, 128), rand(B, H, 128), rand(B, cap, 1, 128)
    k4, v4 = (msa.msa_q4_cache(B, H, cap, "cuda") for _ in range(2))
    kv = [rand(B, cap, H, 128) for _ in range(2)]
    n = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    msa.msa_norm_rope_append(kv, None, None, n, [k4, v4])
    k16, v16 = (msa.msa_q4_read(c, 0, cap) for c in (k4, v4))

    def steps():
        return msa.msa_decode_q4(q, qp, k4, v4, kp, n, top_k, SCALE) + msa.msa_decode(q, qp, k16, v16, kp, n, top_k, SCALE) \
            + msa.msa_window_decode_q4(q, k4, v4, n, 3000, 4, SCALE)
    steps()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = steps()
    for i in range(20):
        q.copy_(rand(B, Hq, 128))
        qp.copy_(rand(B, H, 128))
        kp.copy_(kp.roll(128 * 3 + i, 1))
        n.copy_(torch.randint(1, cap + 1, (B,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        graph.replay()
        got = [x.clone() for x in outs]
        for x, y in zip(got, steps()):
            assert torch.equal(x, y)
