"""Calls of the few-token layer one behind another, each with a route, tokens or
weights that work queued just before it has written to the same buffers."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_group_gemm import gen, random_codes
from test_gpu_moe_few import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# up to 32 pairs and more, with and without clusters, several items per block
@pytest.mark.parametrize("T,H,I,E,k", [(1, 2048, 256, 32, 8), (4, 1024, 1024, 64, 8), (13, 512, 256, 128, 6),
                                       (64, 1024, 512, 32, 4)])
def test_each_call_reads_what_was_queued_before_it(T, H, I, E, k):
    n = 24
    p = problem(T, H, I, E, k, 1)
    g = gen(2)
    logits = torch.randn(n, T, E, generator=g, device=DEV)
    xs = torch.randn(n, T, H, generator=g, device=DEV).to(torch.bfloat16)
    w2 = [p["w2_q"].clone(), random_codes(p["w2_q"].shape, g)]
    idx, w = p["topk_idx"], p["topk_w"]
    want = []
    for i in range(n):  # one at a time
        ep.route(logits[i], k, topk_idx=idx, topk_w=w)
        torch.cuda.synchronize()
        want.append(ep.moe_few(**{**p, "x": xs[i], "w2_q": w2[i % 2]}))
        torch.cuda.synchronize()
    outs = [torch.empty_like(xs[0]) for _ in range(n)]
    workspace = torch.empty(ep.moe_few_workspace_bytes(T, k, I), dtype=torch.uint8, device=DEV)
    for changing in (False, True):
        for i in range(n):  # nothing waits; the route is the kernel right before the layer
            if changing:
                p["w2_q"].copy_(w2[i % 2])
            p["x"].copy_(xs[i])
            ep.route(logits[i], k, topk_idx=idx, topk_w=w)
            q = p if changing else {**p, "w2_q": w2[i % 2]}
            ep.moe_few(**q, out=outs[i], workspace=workspace)
        torch.cuda.synchronize()
        for i in range(n):
            assert torch.equal(outs[i], want[i]), i
