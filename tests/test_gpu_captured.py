"""Training steps through the sparse and dense autograd functions, captured into graphs."""
import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300.inputs import Workload, make_inputs
from tests.parity import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top_k", [3, 0])
def test_graphs_of_one_stream_have_workspaces_of_their_own(top_k):
    """Two graphs captured one after the other, replayed at the same time on two streams, and again after the eager calls'
    workspaces were released and their memory used for something else."""
    w = Workload("captured", B=1, S=1024, Hq=8, Hkv=2, Hp=2, top_k=top_k)
    func = msa.msa_func if top_k else msa.msa_warmup_func
    sets = [make_inputs(w, seed, device="cuda") for seed in (31, 32)]

    def step(g):
        leaves = [g[n].detach().requires_grad_() for n in ("qp", "kp", "q", "k", "v")]
        out, kl = func(*leaves, top_k, w.scale)
        return (out.detach(),) + torch.autograd.grad([out, kl], leaves, [g["dout"], torch.ones_like(kl)])

    msa.clear_workspace_cache()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [[t.clone() for t in step(g)] for g in sets]
        before = {k: t.data_ptr() for k, t in msa._WS_CACHE.items()}
        graphs, outs = [], []
        for g in sets:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs.append(step(g))
            graphs.append(graph)
    torch.cuda.synchronize()
    assert {k: t.data_ptr() for k, t in msa._WS_CACHE.items()} == before  # the captures left the cache alone
    streams = [torch.cuda.Stream() for _ in graphs]

    def replay():
        for _ in range(5):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            for name, a, b in zip(("O", "dqp", "dkp", "dq", "dk", "dv"), got, ref):
                # (fp32 sums in another order: at most a step of bf16 in a few elements)
                close(name, a, b.float(), rel=1e-3, atol=2e-3, ulps=1.0)

    replay()
    msa.clear_workspace_cache()
    torch.cuda.empty_cache()
    filled = [torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    replay()
    del filled
