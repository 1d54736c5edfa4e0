"""Tokens that name an expert several times, with fewer tokens than columns of
a group: the few-token layer against its 64-bit definition."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_group_gemm import gen
from test_gpu_moe_few import check, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def ids(kind, T, k, E, seed):
    if kind == "one":        # every pair to one expert
        idx = torch.full((T, k), E - 1, dtype=torch.int32)
    elif kind == "own":      # every token to an expert of its own, k times
        idx = (torch.arange(T, dtype=torch.int32) % E)[:, None].repeat(1, k)
    else:                    # three experts in any order, some pairs dropped
        g = torch.Generator().manual_seed(seed)
        idx = torch.randint(0, min(3, E), (T, k), generator=g, dtype=torch.int32)
        idx[torch.rand(T, k, generator=g) < 0.15] = -1
    return idx.to(DEV)


# H below 1,024 keeps one block per item; from there few items share theirs
# between 4 or 2 blocks of a cluster
@pytest.mark.parametrize("kind", ["one", "own", "three"])
@pytest.mark.parametrize("T,k", [(1, 2), (1, 8), (1, 32), (2, 2), (2, 8), (3, 6), (5, 2), (5, 32), (7, 8), (8, 4), (9, 8)])
@pytest.mark.parametrize("H,I", [(256, 128), (1024, 128), (2048, 640)])
def test_repeated_experts(kind, T, k, H, I):
    check(problem(T, H, I, 4, k, T * k, ids(kind, T, k, 4, T + k)))


@pytest.mark.parametrize("T,k,H,I", [(1, 8, 7168, 2048), (3, 8, 7168, 256), (1, 2, 16384, 128), (7, 32, 16384, 128)])
def test_repeated_experts_at_the_widest(T, k, H, I):
    check(problem(T, H, I, 2, k, T + H, ids("one", T, k, 2, 1)))


def test_a_repeated_expert_counts_as_often_as_it_is_named():
    # two places of one expert with weights a and b against one place with a + b
    # (exact sums): the same row twice, added in fp32
    p = problem(1, 1024, 256, 8, 2, 5, torch.tensor([[6, 6]], dtype=torch.int32, device=DEV))
    p["topk_w"] = torch.tensor([[0.25, 0.5]], device=DEV)
    one = {**p, "topk_idx": p["topk_idx"][:, :1].contiguous(), "topk_w": torch.tensor([[0.75]], device=DEV)}
    a, b = ep.moe_few(**p).float(), ep.moe_few(**one).float()
    # fl(0.25 y) + 0.5 y is rounded twice, 0.75 y once, then both to bf16
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-30).all()


def test_repeated_experts_give_the_same_bits_every_time():
    g = gen(3)
    p = problem(6, 512, 256, 4, 4, 8, torch.randint(0, 2, (6, 4), generator=g, device=DEV, dtype=torch.int32))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ep.moe_few(**p, status=status)
    assert ep.status_read(status) == 0
    assert torch.equal(out, ep.moe_few(**p))
