"""Tensors that the router's, the products' and the few-token layer's kernels
write to are refused where they lie elsewhere than the inputs."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_moe_few import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def calls():
    """Each call as a function of its status word."""
    p = problem(4, 256, 128, 4, 2, 1)
    rows = torch.zeros(8, 256, dtype=torch.uint8, device=DEV)
    scales = torch.ones(8, 2, device=DEV)
    at = (torch.full((4,), 2, dtype=torch.int32, device=DEV), 2 * torch.arange(5, dtype=torch.int32, device=DEV))
    return {
        "route": lambda s: ep.route(torch.zeros(4, 16, device=DEV), 2, status=s),
        "product": lambda s: ep.group_gemm_fp8(rows, scales, p["w13_q"], p["w13_scale"], *at, status=s),
        "swiglu": lambda s: ep.group_gemm_swiglu_fp8(rows, scales, p["w13_q"], p["w13_scale"], *at, status=s),
        "few": lambda s: ep.moe_few(**p, status=s),
    }


@pytest.mark.parametrize("name", ["route", "product", "swiglu", "few"])
def test_status_words(name):
    call = calls()[name]
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device=DEV),
                torch.zeros(1, dtype=torch.float32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError):
            call(bad)
    for dtype in (torch.int32, torch.uint32):
        word = torch.zeros(1, dtype=dtype, device=DEV)
        call(word)
        assert ep.status_read(word) == 0


def test_workspaces_of_the_few_token_layer():
    p = problem(4, 256, 128, 4, 2, 2)
    need = ep.moe_few_workspace_bytes(4, 2, 128)
    for bad in (torch.zeros(need, dtype=torch.uint8), torch.zeros(2 * need, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            ep.moe_few(**p, workspace=bad)
    ok = torch.zeros(need // 4, dtype=torch.float32, device=DEV)   # any type of that many bytes
    assert torch.equal(ep.moe_few(**p, workspace=ok), ep.moe_few(**p))
