"""Logits and their gradient captured into a graph, replayed on changed histories:
the form in which a CTA reads the lists itself and the one with a table."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

from .test_gpu_logits import bwd_params, check, dev, make, rng

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("N,V,L,K", [(8, 5000, 100, 10), (42, 50257, 300, 20), (42, 50257, 600, 900)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_replay_on_other_histories(N, V, L, K, dtype):
    x, p = make(N, V, dtype, L, L, K, 0.3)
    tables = N * V > 1 << 21
    assert (pkg.ce_logits_workspace_bytes(N, V, dtype, L, K) > 0) == tables
    xd, pd = x.to(DEV), dev(p)
    go = torch.randn(N, V, generator=rng(1)).to(dtype).to(DEV)
    there = xd.clone()
    grad = torch.empty_like(xd)
    for _ in range(2):  # what a first call sets up is not captured
        pkg.ce_logits_process(xd, **pd)
        pkg.ce_logits_process_bwd(go, xd, **bwd_params(pd))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = pkg.ce_logits_process(xd, **pd)
        pkg.ce_logits_process(there, out=there, **pd)
        pkg.ce_logits_process_bwd(go, xd, grad=grad, **bwd_params(pd))
    for seed in (2, 3):
        p["history"] = torch.randint(0, V, (N, L), generator=rng(seed))
        p["history_lengths"] = torch.randint(0, L + 1, (N,), generator=rng(seed + 9))
        pd["history"].copy_(p["history"])
        pd["history_lengths"].copy_(p["history_lengths"])
        there.copy_(xd)
        for t in (y, grad):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(y, x, p)
        check(grad, x, p, go=go)
        assert torch.equal(there, y)
        assert torch.equal(y, pkg.ce_logits_process(xd, **pd))
        assert torch.equal(grad, pkg.ce_logits_process_bwd(go, xd, **bwd_params(pd)))
