"""Long chains of launches: products, elementwise passes and cluster kernels one
behind another and beside each other, the same results every time."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_expert_training import layer_of, problem

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF16)


def test_training_steps_back_to_back():
    p = problem(1000, 512, 256, 16, 4, 1, shared=128, dropped=0.05)
    layer = layer_of(p)

    def step():
        out, saved = layer.forward(p["x"], p["idx"], p["w"])
        return (out,) + tuple(layer.backward(p["dout"], saved))

    want = [v.clone() for v in step()]
    for _ in range(10):
        for _ in range(20):
            got = step()
        assert ep.status_read(layer.status) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_backward_passes_back_to_back():
    """Elementwise pass, input product and weight product in turn, at a size that
    fills the SMs."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    M, N, K = 4096, 2048, 7168
    args = [(normal(g, M, N), normal(g, M, K), normal(g, N, K), normal(g, M, N)) for _ in range(2)]
    dz, dx = torch.empty_like(args[0][0]), torch.empty_like(args[0][1])
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def back(i):
        return ep.linear_backward(*args[i], "gelu", dz=dz, dx=dx, dw=dw, dbias=db, status=status)

    want = [[v.clone() for v in back(i)] for i in range(2)]
    for _ in range(10):
        for i in range(50):
            got = back(i % 2)
        assert ep.status_read(status) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


def test_products_beside_other_kernels():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    dy, x, w, z = normal(g, 1000, 512), normal(g, 1000, 1024), normal(g, 512, 1024), normal(g, 1000, 512)
    y, dout, few = normal(g, 8000, 512), normal(g, 1000, 512), normal(g, 4, 1024)
    idx = torch.rand(1000, 64, generator=g, device=DEV).topk(8, 1).indices.int()
    tw = torch.rand(1000, 8, generator=g, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def products():
        return ep.linear_backward(dy, x, w, z, "gelu", status=status)

    def others():
        lay = ep.layout(idx, 64)
        return (ep.combine(y, tw, lay.dst_row), ep.combine_backward(dout, y, tw, lay.dst_row)[1],
                ep.linear(few, w, status=status)) + tuple(products())

    want, also = products(), others()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for _ in range(20):
            with torch.cuda.stream(a):
                one = products()
            with torch.cuda.stream(b):
                two = others()
        torch.cuda.synchronize()
        assert ep.status_read(status) == 0
        assert all(torch.equal(u, v) for u, v in zip(one, want)) and all(torch.equal(u, v) for u, v in zip(two, also))


def test_gradients_of_rows_in_parts_back_to_back():
    """The elementwise pass, both products and the pass over the parts' sums, called
    and as one graph replayed, on two streams with a workspace each."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    M, N, K = 8192, 256, 1032
    dy, x, w, z = normal(g, M, N), normal(g, M, K), normal(g, N, K), normal(g, M, N)
    assert ep.linear_backward_workspace_bytes(M, K, N, "silu") > 0
    want = ep.linear_backward(dy, x, w, z, "silu")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            ws = torch.empty(ep.linear_backward_workspace_bytes(M, K, N, "silu"), dtype=torch.uint8, device=DEV)
            out = ep.linear_backward(dy, x, w, z, "silu", workspace=ws)
            outs.append((ws, out))
    for _ in range(300):
        for st, (ws, out) in zip(streams, outs):
            with torch.cuda.stream(st):
                ep.linear_backward(dy, x, w, z, "silu", dz=out.dz, dx=out.dx, dw=out.dw, dbias=out.dbias, workspace=ws)
    torch.cuda.synchronize()
    for _, out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [ep.linear_backward(dy, x, w, z, "silu") for _ in range(4)]
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
