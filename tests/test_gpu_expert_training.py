"""A whole expert layer forward and backward through the package's calls against
the same layer in 64 bits, whose gradients autograd forms."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def problem(T, H, I, E, k, seed, shared=0, dropped=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, amp=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * amp).to(BF16)

    p = dict(x=normal(T, H), dout=normal(T, H), w13=normal(E, 2 * I, H, amp=H ** -0.5), w2=normal(E, H, I, amp=I ** -0.5))
    p["idx"] = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.int()
    p["idx"][torch.rand(T, k, generator=g, device=DEV) < dropped] = -1
    p["w"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
    if shared:
        p["s13"], p["s2"] = normal(2 * shared, H, amp=H ** -0.5), normal(H, shared, amp=shared ** -0.5)
    return p


def layer_of(p):
    return ep.TrainableExpertLayer(p["w13"], p["w2"], p.get("s13"), p.get("s2"))


def definition(p):
    """(out, gradients of x, w, w13, w2, s13, s2) in 64 bits."""
    leaves = {n: p[n].double().requires_grad_() for n in ("x", "w", "w13", "w2", "s13", "s2") if n in p}

    def gated(v, w13, w2):
        g, u = (v @ w13.T).chunk(2, -1)
        return (torch.nn.functional.silu(g) * u) @ w2.T

    x = leaves["x"]
    out = torch.zeros_like(x)
    for e in range(p["w13"].shape[0]):
        t, j = torch.nonzero(p["idx"] == e, as_tuple=True)
        if t.numel():
            out = out.index_add(0, t, leaves["w"][t, j, None] * gated(x[t], leaves["w13"][e], leaves["w2"][e]))
    if "s13" in p:
        out = out + gated(x, leaves["s13"], leaves["s2"])
    out.backward(p["dout"].double())
    return out.detach(), {n: v.grad for n, v in leaves.items()}


# A chain of n bf16 roundings, each of independent values off by at most 2^-8
# (2^-9 on average, uniformly), moves a result that sums many of them by less
# than 2^-8 sqrt(n) of its norm; the last one itself counts among them.  out: h,
# y, out (z is rounded for the backward pass alone).  dx: z, dy, dz, drows, dx
# and the shared expert's sum.  dw: y or (h, dy), (z, dy, dz).
def near(got, want, roundings):
    return (got.double() - want).norm() <= 2.0 ** -8 * roundings ** 0.5 * want.norm() + 1e-30


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 16, 4, 2), (7, 136, 48, 8, 3), (200, 256, 128, 8, 4), (300, 512, 272, 16, 2),
                                       (1000, 128, 64, 4, 4)])
@pytest.mark.parametrize("shared", [0, 48])
def test_forward_and_gradients(T, H, I, E, k, shared):
    p = problem(T, H, I, E, k, T, shared, dropped=0.1)
    layer = layer_of(p)
    out, saved = layer.forward(p["x"], p["idx"], p["w"])
    got = layer.backward(p["dout"], saved)
    assert ep.status_read(layer.status) == 0
    want, grads = definition(p)
    assert near(out, want, 4)
    assert near(got.dx, grads["x"], 7)
    assert near(got.dtopk_w, grads["w"], 3)
    assert near(got.dw13, grads["w13"], 5) and near(got.dw2, grads["w2"], 3)
    if shared:
        assert near(got.dshared13, grads["s13"], 5) and near(got.dshared2, grads["s2"], 3)
    assert (got.dtopk_w[p["idx"] < 0] == 0).all()
    idle = torch.bincount(p["idx"][p["idx"] >= 0].long(), minlength=E) == 0
    assert (got.dw13[idle] == 0).all() and (got.dw2[idle] == 0).all()


def test_gradients_are_added():
    p = problem(60, 128, 64, 8, 2, 1, shared=32)
    layer = layer_of(p)
    _, saved = layer.forward(p["x"], p["idx"], p["w"])
    once = layer.backward(p["dout"], saved)
    first = [once.dw13.clone(), once.dw2.clone(), once.dshared13.clone(), once.dshared2.clone()]
    twice = layer.backward(p["dout"], saved, grads=once)
    for a, b, c in zip(first, twice[2:], once[2:]):
        assert b is c and torch.equal(b, 2 * a)  # v + v is exact
    half = layer.backward(p["dout"], saved, dtype=BF16)
    assert all(h.dtype is BF16 and near(h, f.double(), 1) for h, f in zip(half[2:], first))


def test_a_route_without_experts():
    p = problem(5, 64, 16, 4, 2, 2)
    p["idx"].fill_(-1)
    layer = layer_of(p)
    out, saved = layer.forward(p["x"], p["idx"], p["w"])
    got = layer.backward(p["dout"], saved)
    assert (out == 0).all() and all((g == 0).all() for g in got[:4])


def test_no_tokens():
    p = problem(3, 64, 16, 4, 2, 6, shared=16)
    layer = layer_of(p)
    out, saved = layer.forward(p["x"][:0], p["idx"][:0], p["w"][:0])
    got = layer.backward(p["dout"][:0], saved)
    assert out.shape == (0, 64) and got.dx.shape == (0, 64) and got.dtopk_w.shape == (0, 2)
    assert all((g == 0).all() for g in got[2:]) and ep.status_read(layer.status) == 0


def test_captured_step():
    """Forward and backward in one graph, replayed on other inputs."""
    p, q = problem(90, 128, 64, 8, 2, 3, shared=32), problem(90, 128, 64, 8, 2, 4, shared=32)
    layer = layer_of(p)

    def step():
        out, saved = layer.forward(p["x"], p["idx"], p["w"])
        return (out,) + tuple(layer.backward(p["dout"], saved))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        got = step()
    for n in ("x", "dout", "idx", "w"):
        p[n].copy_(q[n])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert ep.status_read(layer.status) == 0


def test_refusals():
    p = problem(4, 64, 16, 4, 2, 5, shared=16)
    for bad in ((p["w13"], p["w2"][:, :32]), (p["w13"][:2], p["w2"]), (p["w13"], p["w2"], p["s13"]),
                (p["w13"], p["w2"], p["s13"], p["s2"][:, :8])):
        with pytest.raises(ValueError):
            ep.TrainableExpertLayer(*bad)
    layer = layer_of(p)
    for bad in ((p["x"][:, :32], p["idx"], p["w"]), (p["x"], p["idx"][:2], p["w"][:2]), (p["x"], p["idx"], p["w"][:, :1])):
        with pytest.raises(ValueError):
            layer.forward(*bad)
    _, saved = layer.forward(p["x"], p["idx"], p["w"])
    with pytest.raises(ValueError):
        layer.backward(p["dout"][:2], saved)
