"""Attention over packed sequences on the GPU, each sequence against the plain 64-bit form with its counted roundings."""
import random

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain
from tests.plain_local import check

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def make(seed, rows, Hq, Hkv, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = [torch.randn((rows, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq)]
    for t in out:  # what lies behind the last sequence may be anything
        if pad:
            t[rows - pad:] = float("nan")
    return out


def against_plain(lengths, q, k, v, got, window, which=None, dout=None):
    """got: o, lse and, with dout, dq, dk, dv."""
    at = 0
    for i, n in enumerate(lengths):
        s = slice(at, at + n)
        at += n
        if n == 0 or (which is not None and i not in which):
            continue
        want = plain.window(q[None, s], k[None, s], v[None, s], window, 0, SCALE, None if dout is None else dout[None, s])
        for name, t in zip(("o", "lse", "dq", "dk", "dv"), got):
            check(f"{name} of sequence {i}", t[:, s][None] if name == "lse" else t[None, s], want[name])
    o, lse = got[:2]
    assert (o[at:] == 0).all() and (lse[:, at:] == -torch.inf).all()
    for t in got[2:]:
        assert (t[at:] == 0).all()


def run(lengths, Hq, Hkv, pad=0, window=None, seed=0, train=True, which=None):
    rows = sum(lengths) + pad
    q, k, v, dout = make(seed, rows, Hq, Hkv, pad)
    plan = msa.msa_packed_plan(lengths, Hq, Hkv, rows=rows, window=window, device="cuda")
    ws = torch.full((plan.workspace_size(msa.OP_PACKED_BACKWARD),), 255, dtype=torch.uint8, device="cuda")
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE, ws=ws)
    assert msa.msa_device_status(ws) == 0
    got = (o, lse)
    if train:
        ws.fill_(255)
        got += msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE, ws=ws)
        assert msa.msa_device_status(ws) == 0
    against_plain(lengths, q, k, v, got, rows if window is None else window, which, dout if train else None)
    return plan


@pytest.mark.parametrize("lengths,Hq,Hkv,pad,window", [
    ([1], 1, 1, 0, None), ([1, 1, 1], 16, 1, 2, None), ([2, 0, 1, 3], 8, 2, 0, None), ([128], 2, 2, 0, None), ([127, 129, 128], 8, 8, 0, None),
    ([300, 1, 0, 77, 513], 8, 2, 5, None), ([40] * 20, 16, 4, 1, None), ([1000], 4, 1, 24, None), ([5, 900, 5], 16, 1, 0, None),
    ([700, 20, 300], 8, 1, 3, 128), ([700, 20, 300], 8, 4, 0, 1), ([64, 1, 640, 33], 2, 1, 0, 100), ([17] * 9 + [400], 1, 1, 7, 33),
    ([255, 257], 64, 8, 0, None), ([3, 1200, 2, 800], 32, 8, 1, 500),
])
def test_against_plain(lengths, Hq, Hkv, pad, window):
    run(lengths, Hq, Hkv, pad, window, seed=len(lengths) + Hq)


@pytest.mark.parametrize("seed", range(6))
def test_drawn(seed):
    r = random.Random(seed)
    Hkv = r.choice([1, 2, 4])
    Hq = Hkv * r.choice([1, 2, 4, 8, 16])
    lengths = [r.choice([0, 1, 16, 128, r.randint(1, 60), r.randint(1, 900)]) for _ in range(r.randint(1, 12))] + [r.randint(1, 50)]
    run(lengths, Hq, Hkv, r.choice([0, 1, 130]), r.choice([None, None, 1, 64, 200]), seed)


def test_split_key_blocks():
    """One long sequence of one KV head: every key block's query tiles are several items, whose partials are joined."""
    plan = run([2500, 40], 8, 1)
    assert plan.counts.slots > 0 and plan.counts.joins > 0
    plan = run([2500, 40], 1, 1, window=700)
    assert plan.counts.joins > 0


def test_more_sequences_than_a_launch_takes():
    r = random.Random(5)
    lengths = [r.randint(0, 5) for _ in range(2500)]
    which = {0, 1, 2, 3, 4, 957, 958, 959, 960, 961, 962, 1918, 1919, 1920, 1921, 1922, 2495, 2496, 2497, 2498, 2499}
    run(lengths, 8, 2, 3, which=which)


def test_no_sequence():
    for lengths in ([], [0, 0]):
        q, k, v, dout = make(0, 5, 8, 2, 5)
        plan = msa.msa_packed_plan(lengths, 8, 2, rows=5, device="cuda")
        ws = torch.full((plan.workspace_size(msa.OP_PACKED_BACKWARD),), 255, dtype=torch.uint8, device="cuda")
        o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE, ws=ws)
        assert msa.msa_device_status(ws) == 0
        grads = msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE, ws=ws)
        assert msa.msa_device_status(ws) == 0
        assert (o == 0).all() and (lse == -torch.inf).all() and all((g == 0).all() for g in grads)


def test_lengths_as_a_tensor():
    q, k, v, _ = make(1, 300, 8, 2)
    a = msa.msa_packed_plan(torch.tensor([100, 200], dtype=torch.int32), 8, 2, device=q.device)
    b = msa.msa_packed_plan([100, 200], 8, 2, device="cuda")
    for x, y in zip(msa.msa_packed_forward(q, k, v, a, SCALE), msa.msa_packed_forward(q, k, v, b, SCALE)):
        assert torch.equal(x, y)
    with pytest.raises(msa.MSAError, match="host"):
        msa.msa_packed_plan(torch.tensor([100, 200], device="cuda"), 8, 2)


def test_values_that_are_not_finite_stay_in_their_sequence():
    lengths = [30, 50, 200, 40]
    q, k, v, _ = make(2, 320, 8, 2)
    plan = msa.msa_packed_plan(lengths, 8, 2, device="cuda")
    clean = msa.msa_packed_forward(q, k, v, plan, SCALE)
    v[79] = float("nan")  # the second's last row
    v[281] = float("inf")  # the last's second
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    assert torch.equal(lse, clean[1])
    rows = [r for r in range(320) if r != 79 and not r >= 281]
    for name, x in (("o", o[rows]),):
        assert torch.isfinite(x).all()
        # rows that are computed again round P differently
        assert (x.float() - clean[0][rows].float()).abs().max() <= 2 ** -6
    assert not torch.isfinite(o[79]).any() and not torch.isfinite(o[281:]).any()
    k[100] = float("nan")  # the third's 21st key: no row of another sequence
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    keep = [r for r in rows if not 100 <= r < 280]
    assert torch.isfinite(o[keep]).all() and torch.isfinite(lse[:, keep]).all()


def test_same_bits_every_time():
    lengths = [700, 3, 1500, 90, 1]
    q, k, v, dout = make(3, sum(lengths), 16, 4)
    def once():
        plan = msa.msa_packed_plan(lengths, 16, 4, device="cuda")
        o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
        return (o, lse) + msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE)
    a = once()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, once()))


def test_as_a_batch_of_one_length():
    """Sequences of one length are the window operator's batch."""
    B, S = 3, 200
    q, k, v, dout = make(4, B * S, 8, 2)
    plan = msa.msa_packed_plan([S] * B, 8, 2, window=60, device="cuda")
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    b = lambda x: x.view(B, S, -1, 128)  # noqa: E731
    o2, lse2 = msa.msa_window_forward(b(q), b(k), b(v), 60, 0, SCALE)
    assert (o.float() - o2.flatten(0, 1).float()).abs().max() <= 2 ** -6
    assert (lse.view(8, B, S).transpose(0, 1) - lse2).abs().max() <= plain.F


def test_autograd_and_differences():
    lengths, rows = [60, 1, 100], 170
    q, k, v, dout = make(5, rows, 4, 2)
    plan = msa.msa_packed_plan(lengths, 4, 2, rows=rows, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = msa.msa_packed_func(*leaves, plan, SCALE)
    o.backward(dout)
    got = [t.grad for t in leaves]
    _, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    against_plain(lengths, q, k, v, (o.detach(), lse, *got), rows, dout=dout)

    def loss(q, k, v):
        total, at = 0.0, 0
        for n in lengths:
            s = slice(at, at + n)
            at += n
            x = plain.window(q[None, s], k[None, s], v[None, s], rows, 0, SCALE)["o"][0]
            total = total + (x[0] * dout[s].double()).sum()
        return total

    h = 1e-6
    for i, g in enumerate(got):
        d = torch.randn(g.shape, device="cuda", dtype=torch.float64)
        at = [t.double() for t in (q, k, v)]
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + h * d, at[i] - h * d
        want = (loss(*plus) - loss(*minus)) / (2 * h)
        have = (g.double() * d).sum()
        # each gradient's own bound, summed over the direction, and the difference's error
        bound, a = 0.0, 0
        for n in lengths:
            s = slice(a, a + n)
            a += n
            e = plain.window(q[None, s], k[None, s], v[None, s], rows, 0, SCALE, dout[None, s])[("dq", "dk", "dv")[i]][1]
            bound = bound + (e[0] * d[s].abs()).sum()
        assert abs(have - want) <= bound + 1e-3


def test_captured_with_its_plan_while_an_eager_graph_lives():
    """A training step, plan included, captured and replayed over new tensors while an eager graph of other leaves of
    the same tensors is alive; another stream than the default."""
    lengths, rows = [90, 200, 5], 300
    q, k, v, dout = make(6, rows, 8, 2, 5)
    eager = [t.clone().nan_to_num(0.0).requires_grad_() for t in (q, k, v)]
    keep = msa.msa_packed_func(*eager, msa.msa_packed_plan(lengths, 8, 2, rows=rows, device="cuda"), SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        plan = msa.msa_packed_plan(lengths, 8, 2, rows=rows, device="cuda")
        o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
        return (o, lse) + msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE)

    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        for seed in (7, 8):
            new = make(seed, rows, 8, 2, 5)
            for t, n in zip((q, k, v, dout), new):
                t.copy_(n)
            graph.replay()
            side.synchronize()
            against_plain(lengths, q, k, v, out, rows, dout=dout)
    torch.cuda.current_stream().wait_stream(side)
    keep.backward(torch.ones_like(keep))
    assert all(torch.isfinite(t.grad).all() for t in eager)


def test_one_plan_for_several_layers_on_a_stream_of_its_own():
    lengths = [100, 300]
    side = torch.cuda.Stream()
    plan = msa.msa_packed_plan(lengths, 8, 2, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for seed in (1, 2):
        q, k, v, dout = make(seed, 400, 8, 2)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
            got = (o, lse) + msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE)
        side.synchronize()
        against_plain(lengths, q, k, v, got, 400, dout=dout)


def test_arguments_refused():
    q, k, v, dout = make(9, 50, 8, 2)
    plan = msa.msa_packed_plan([50], 8, 2, device="cuda")
    with pytest.raises(msa.MSAError, match="shape"):
        msa.msa_packed_forward(q[:40], k, v, plan, SCALE)
    with pytest.raises(msa.MSAError, match="shape"):
        msa.msa_packed_forward(q, k[:, :1].contiguous(), v, plan, SCALE)
    with pytest.raises(msa.MSAError, match="bfloat16"):
        msa.msa_packed_forward(q.float(), k, v, plan, SCALE)
    with pytest.raises(msa.MSAError, match="contiguous"):
        msa.msa_packed_forward(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, plan, SCALE)
    with pytest.raises(msa.MSAError, match="invalid argument"):
        msa.msa_packed_forward(q, k, v, plan, 0.0)
    with pytest.raises(msa.MSAError, match="too small"):
        msa.msa_packed_forward(q, k, v, plan, SCALE, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(msa.MSAError, match="Hq / Hkv"):
        msa.msa_packed_plan([50], 9, 2, device="cuda")
    with pytest.raises(msa.MSAError, match="window"):
        msa.msa_packed_plan([50], 8, 2, window=0, device="cuda")


def test_tensors_past_2_31_elements():
    """A million tokens of 20 heads: the last sequences lie behind 2^31 elements of q, and of lse's last row."""
    rows, Hq, Hkv = 1 << 20, 20, 20
    r = random.Random(1)
    lengths, left = [], rows - 3
    while left:
        n = min(left, r.randint(1, 400))
        lengths.append(n)
        left -= n
    last = len(lengths)
    q, k, v, dout = make(10, rows, Hq, Hkv, 3)
    assert q.numel() > 2 ** 31
    plan = msa.msa_packed_plan(lengths, Hq, Hkv, rows=rows, device="cuda")
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    got = (o, lse) + msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE)
    against_plain(lengths, q, k, v, got, rows, which={0, 1, last // 2, last - 3, last - 2, last - 1}, dout=dout)


def test_lengths_of_every_kind():
    """Lengths as a list, a tuple, a range, a host tensor, an iterator, floats without a fraction: one plan."""
    lens = [3, 0, 200, 17, 1]
    want = run_forward(lens)
    for kind in (tuple(lens), torch.tensor(lens), torch.tensor(lens, dtype=torch.int32), iter(lens), [float(n) for n in lens]):
        for x, y in zip(want, run_forward(kind)):
            assert torch.equal(x, y)
    assert msa.msa_packed_plan(range(4), 2, 1, device="cuda").rows == 6
    for bad in ([-1], [5, -2 ** 31], [2 ** 31], [2 ** 40, 1], [-2 ** 40], [1.0, -3.0]):
        with pytest.raises(msa.MSAError, match="lengths must be in"):
            msa.msa_packed_plan(bad, 2, 1, device="cuda")


def run_forward(lengths):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randn((221, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    k, v = torch.randn((2, 221, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    return msa.msa_packed_forward(q, k, v, msa.msa_packed_plan(lengths, 4, 2, device="cuda"), 0.1)


@pytest.mark.parametrize("train", [False, True])
def test_a_plan_dropped_while_another_stream_reads_its_table(train):
    """Planned on one stream, used on another, dropped before that one has come to it: the table's memory is given to nobody
    until it has."""
    lengths, Hq, Hkv = [700, 3, 1500, 90], 8, 2
    q, k, v, dout = make(11, sum(lengths), Hq, Hkv)
    plan = msa.msa_packed_plan(lengths, Hq, Hkv, device="cuda")
    o, lse = msa.msa_packed_forward(q, k, v, plan, SCALE)
    want = (o, lse) + (msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE) if train else ())
    torch.cuda.synchronize()
    plan = msa.msa_packed_plan(lengths, Hq, Hkv, device="cuda")
    at, size = plan.table.data_ptr(), plan.table.numel()
    compute = torch.cuda.Stream()
    compute.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(compute):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        if train:
            got = (o, lse) + msa.msa_packed_backward(q, k, v, o, lse, dout, plan, SCALE)
        else:
            got = msa.msa_packed_forward(q, k, v, plan, SCALE)
    del plan
    held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(50)]
    busy = not compute.query()
    assert busy and all(t.data_ptr() != at for t in held)
    for t in held:
        t.fill_(255)
    compute.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
