"""Infinities and NaN in rows that a query of the window attention does not see: none reaches it."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from tests import plain_local as plain
from tests.test_gpu_window import DEV, SCALE, forward, tensors

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def check_rows(q, k, v, bad, W, ns):
    """bad [B, S]: tokens whose K and V rows are not finite.  Queries that see none of them against the plain form
    without them, the others not finite."""
    o, lse = forward(q, k, v, W, ns)
    B, S, Hq, _ = q.shape
    sees = torch.einsum("tj,bj->bt", plain.visible(S, W, ns, DEV).float(), bad.float()) > 0
    clean = [torch.where(bad[..., None, None], torch.zeros_like(x), x) for x in (k, v)]
    own = torch.where(torch.isfinite(q).all(-1, keepdim=True).all(-2, keepdim=True), q, torch.zeros_like(q))
    want = plain.window(own, *clean, W, ns, SCALE)
    kept = ~sees & torch.isfinite(q).flatten(2).all(-1)
    assert kept.any()
    plain.check("o", o[kept], tuple(x[kept] for x in want["o"]))
    plain.check("lse", lse.transpose(1, 2)[kept], tuple(x.transpose(1, 2)[kept] for x in want["lse"]))
    assert not torch.isfinite(o[sees]).flatten(1).all(-1).any()
    return o


@pytest.mark.parametrize("Hq,Hkv,W,ns", [(8, 2, 64, 0), (8, 8, 300, 4), (16, 1, 40, 20), (4, 2, 2 ** 20, 0), (16, 2, 1, 0)])
def test_padding_is_anything(Hq, Hkv, W, ns):
    """A ragged batch: what stands behind a sequence's last token (as uninitialised memory may) is not seen by it."""
    lens = [300, 130, 1, 257]
    q, k, v, _ = tensors(4, 300, Hq, Hkv, seed=70)
    bad = torch.arange(300, device=DEV) >= torch.tensor(lens, device=DEV)[:, None]
    for x, value in ((q, NAN), (k, INF), (v, NAN)):
        x[bad] = value
    check_rows(q, k, v, bad, W, ns)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 4), (8, 2), (16, 2), (32, 2)])
@pytest.mark.parametrize("W,ns", [(5, 0), (130, 3), (200, 130)])
@pytest.mark.parametrize("value", [NAN, -INF])
def test_single_rows(Hq, Hkv, W, ns, value):
    """Rows in the middle: the queries in front of them, and those whose window has left them behind, share tiles
    with queries that see them.  The last of three sequences has none."""
    q, k, v, _ = tensors(3, 700, Hq, Hkv, seed=71)
    bad = torch.zeros(3, 700, dtype=torch.bool, device=DEV)
    bad[0, [300, 431]] = True
    bad[1, [ns + 1, 512, 699]] = True  # beside the sinks, at a tile's start, the last token
    v[bad] = value
    o = check_rows(q, k, v, bad, W, ns)
    clean, _ = forward(q[2:], k[2:], v[2:], W, ns)
    assert (o[2:] - clean).float().abs().max() <= 2 ** -6 * clean.float().abs().max()


def test_one_element_of_one_head():
    """One infinite element of one KV head: the other heads, and the queries that do not see it, are finite."""
    q, k, v, _ = tensors(2, 5000, 64, 8, seed=72)
    want, _ = forward(q, k, v, 300, 4)
    v[1, 2500, 3, 17] = INF
    o, lse = forward(q, k, v, 300, 4)
    t = torch.arange(5000, device=DEV)
    sees = (t >= 2500) & (t < 2800)
    hit = ~torch.isfinite(o).all(-1)
    assert hit[1, sees, 24:32].all() and int(hit.sum()) == 300 * 8
    ok = ~hit
    e = plain.HALF * 2 + plain.F  # both round P and the result
    assert ((o - want)[ok].float().abs() <= 2 * e * v[torch.isfinite(v)].float().abs().max()).all()


def test_every_row_not_finite():
    """A run that has diverged: every output says so, at no great cost."""
    q, k, v, _ = tensors(1, 4096, 32, 4, seed=73)
    v.fill_(NAN)
    o, _ = forward(q, k, v, 1000, 4)
    assert torch.isnan(o).all()


@pytest.mark.parametrize("what", ["q", "k", "huge"])
def test_diverged_inputs_cost_no_walk(what):
    """Rows whose own scores are not finite, or that overflow with nothing unseen in their tiles, are not computed again:
    a long dense call stays within five times a finite one's time (their walks, a warp a row, would take hundreds)."""
    q, k, v, _ = tensors(1, 32768, 16, 2, seed=75)

    def ms():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        msa.msa_window_forward(q, k, v, 2 ** 30, 0, SCALE)
        a.record()
        for _ in range(3):
            msa.msa_window_forward(q, k, v, 2 ** 30, 0, SCALE)
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    clean = ms()
    if what == "huge":
        v.fill_(3e38)
        q.mul_(4)  # row maxima that move: O is held relative to an earlier one
    else:
        (q if what == "q" else k).fill_(NAN)
    assert ms() <= 5 * clean


@pytest.mark.parametrize("ns", [1, 125, 131])
def test_rows_beside_the_sinks(ns):
    """Sinks are loaded in eights: the rows up to the next multiple reach no later query (125: within a whole tile)."""
    q, k, v, _ = tensors(1, 3000, 16, 2, seed=76)
    bad = torch.zeros(1, 3000, dtype=torch.bool, device=DEV)
    bad[0, ns:ns + 2] = True
    k[bad], v[bad] = NAN, NAN
    check_rows(q, k, v, bad, 200, ns)
    n = torch.tensor([3000], dtype=torch.int32, device=DEV)
    o, _ = msa.msa_window_decode(q[:, -1].contiguous(), k, v, n, 200, ns, SCALE)
    assert torch.isfinite(o).all()


def test_captured_and_autograd():
    q, k, v, do = tensors(2, 200, 8, 2, seed=74)
    want, _ = forward(q, k, v, 50, 4)
    k[:, 150:], v[:, 150:] = NAN, NAN
    o = msa.msa_window_func(q, k, v, 50, 4, SCALE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2 = msa.msa_window_func(q, k, v, 50, 4, SCALE)
    graph.replay()
    ref = plain.window(q[:, :150], k[:, :150], v[:, :150], 50, 4, SCALE)["o"]
    for x in (o, o2, want):
        plain.check("o", x[:, :150], ref)
