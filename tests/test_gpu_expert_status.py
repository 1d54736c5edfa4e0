"""The expert layer's status word under calls on several streams, and the call
that joins two words."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_expert_layer import layer_of
from test_gpu_moe_few import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_flags_of_one_stream_survive_the_calls_of_another():
    """Clean calls of the longer path on one stream, beside them calls that raise
    a flag and look for it on another, again and again."""
    p, few = problem(100, 256, 128, 8, 2, 1), problem(4, 256, 128, 8, 2, 2)
    layer = layer_of(p, 2)
    assert not layer.few(100) and layer.few(4)
    bad = few["topk_idx"].clone()
    bad[1, 0] = 99
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    layer.experts(p["x"], p["topk_idx"], p["topk_w"])
    layer.experts(few["x"], bad, few["topk_w"])
    torch.cuda.synchronize()
    clean = torch.cuda.CUDAGraph()
    with torch.cuda.graph(clean, stream=a):
        for _ in range(20):
            layer.experts(p["x"], p["topk_idx"], p["topk_w"])
    lost = 0
    for i in range(1000):
        layer.status.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            clean.replay()
        with torch.cuda.stream(b):
            torch.cuda._sleep(1 + i * 613 % 500000)  # somewhere among the clean calls
            layer.experts(few["x"], bad, few["topk_w"])
        torch.cuda.synchronize()
        lost += layer.status.item() != ep.EP_FLAG_BAD_EXPERT
    assert lost == 0


def test_merge_of_two_words():
    word = lambda v, dt=torch.int32: torch.tensor([v], dtype=dt, device=DEV)  # noqa: E731
    into = word(5)
    ep.status_merge(word(0), into)
    assert ep.status_read(into) == 5
    ep.status_merge(word(18), into)
    assert ep.status_read(into) == 23
    for src, dst in ((torch.zeros(1, dtype=torch.int32), into), (word(1, torch.int64), into), (word(1), word(1, torch.uint8))):
        with pytest.raises(ValueError):
            ep.status_merge(src, dst)
    assert ep.status_read(into) == 23
