"""The BF16 products, the dense layer and the gradients inside graph capture as
their very first use, in a fresh process, and captured graphs that are replayed
on two streams at once."""
import os
import subprocess
import sys

import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import sys, torch
sys.path.insert(0, ROOT_DIR)
import combine_ep_layout_02_gb300 as ep
dev = torch.device("cuda:0")
torch.manual_seed(0)
def R(*s):
    return torch.randn(*s, device=dev).to(torch.bfloat16)
E, N, K, per = 3, 96, 64, 40
cnt = torch.full((E,), per, dtype=torch.int32, device=dev)
off = torch.arange(E + 1, dtype=torch.int32, device=dev) * per
x, w, dy, z = R(E * per, K), R(E, N, K), R(E * per, N), R(E * per, 2 * K)
a, b = R(200, 7168), R(256, 7168)
idx = torch.rand(50, 8, device=dev).topk(2, 1).indices.int()
lay = ep.layout(idx, 8)
y, dout, tw = R(100, 64), R(50, 64), torch.rand(50, 2, device=dev)
calls = [lambda: ep.group_gemm(x, w, cnt, off), lambda: ep.group_gemm_swiglu(x, w, cnt, off),
         lambda: ep.group_gemm_dgrad(dy, w, cnt, off), lambda: ep.group_gemm_swiglu_dgrad(dy, w, z, cnt, off),
         lambda: ep.group_gemm_wgrad(dy, x, cnt, off), lambda: ep.group_gemm_wgrad(dy, x, cnt, off, dtype=torch.bfloat16),
         lambda: ep.linear(a, b), lambda: ep.linear(a, b, dtype=torch.float32), lambda: ep.linear(a[:4].contiguous(), b),
         lambda: ep.linear_backward(R0, a, b, Z0, "gelu")[2], lambda: ep.combine_backward(dout, y, tw, lay.dst_row)[0]]
R0, Z0 = R(200, 256), R(200, 256)
torch.cuda.synchronize()
for i, call in enumerate(calls):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        got = call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, call()), i
print("CAPTURE-FIRST OK")
'''


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_first_calls_inside_graph_capture():
    r = subprocess.run([sys.executable, "-c", SCRIPT.replace("ROOT_DIR", repr(ROOT))], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "CAPTURE-FIRST OK" in r.stdout


def test_split_sums_of_two_streams_at_once():
    """Products whose summed index is split hold fp32 parts in a workspace: each
    call has its own."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.randn(256, 7168, generator=g, device=DEV).to(torch.bfloat16)
    xs = [torch.randn(100, 7168, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    assert ep.linear_workspace_bytes(100, 7168, 256) > 0
    want = [ep.linear(x, w) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(50):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(ep.linear(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_a_workspace_that_is_too_small_is_refused():
    x, w = torch.zeros(100, 7168, dtype=torch.bfloat16, device=DEV), torch.zeros(256, 7168, dtype=torch.bfloat16, device=DEV)
    need = ep.linear_workspace_bytes(100, 7168, 256)
    ep.linear(x, w, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    with pytest.raises(ep.EpError):
        ep.linear(x, w, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        ep.linear(x, w, workspace=torch.empty(need, dtype=torch.uint8))


def test_the_current_stream_orders_the_calls():
    """A call on a side stream sees what that stream wrote before it."""
    x, w = torch.zeros(64, 512, dtype=torch.bfloat16, device=DEV), torch.ones(512, 512, dtype=torch.bfloat16, device=DEV)
    big = torch.zeros(1 << 28, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big.add_(1)          # a millisecond of work in front
        x.fill_(1)
        out = ep.linear(x, w, dtype=torch.float32)
        few = ep.linear(x[:8], w, dtype=torch.float32)
    s.synchronize()
    assert (out == 512).all() and (few == 512).all()
