"""The dense layer, its gradients and the combine's gradient against plain
64-bit definitions."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import product_reference as ref
from gpu_helpers import DEV
from test_gpu_products import BF16, FREE, full, gen, values

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def problem(M, N, K, act, seed, exact=False):
    g = gen(seed)
    n = 2 * N if act == "swiglu" else N
    w = values((n, K), g, exact)
    return dict(x=values((M, K), g, exact), w=w if exact else (w.float() * K ** -0.5).to(BF16), activation=act), g, n


def check(p, bias=None, residual=None, dtype=BF16, keep=False):
    M, n = p["x"].shape[0], p["w"].shape[0]
    N = n // 2 if p["activation"] == "swiglu" else n
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    z = full((M, n)) if keep else None
    out = ep.linear(**p, bias=bias, residual=residual, out=full((M, N), dtype), z=z, status=status)
    assert ep.status_read(status) == 0
    want, off, y, dy = ref.linear(p["x"], p["w"], bias, p["activation"], residual)
    assert ref.close(out, want, off)
    if keep:
        assert ref.close(z, y, dy)
    again = ep.linear(**p, bias=bias, residual=residual, dtype=dtype)
    assert torch.equal(out, again)  # the order of every sum is fixed


MS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 257, 513]


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("N,K", [(8, 8), (256, 2048), (136, 264), (1000, 1032), (48, 7168), (16, 64)])
def test_plain_products_are_exact_on_exact_data(M, N, K):
    p, g, n = problem(M, N, K, "none", 1, exact=True)
    want = ref.product(p["x"], p["w"])[0]
    assert torch.equal(ep.linear(**p), want.to(BF16))
    assert torch.equal(ep.linear(**p, dtype=torch.float32), want.float())
    bias, res = values((n,), g, True), values((M, n), g, True)
    assert torch.equal(ep.linear(**p, bias=bias, residual=res), (want + bias.double() + res.double()).to(BF16))


@pytest.mark.parametrize("M", [40, 100, 300])
@pytest.mark.parametrize("K", [504, 512, 520, 576, 1024, 1088, 4104])
def test_float32_sums_in_parts_are_exact(M, K):
    p, g, n = problem(M, 264, K, "none", 14, exact=True)
    assert torch.equal(ep.linear(**p, dtype=torch.float32), ref.product(p["x"], p["w"])[0].float())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 5, 8, 16, 19, 40, 64, 130, 300])
@pytest.mark.parametrize("N,K", [(16, 8), (256, 1024), (400, 136), (144, 2056)])
def test_epilogues(act, M, N, K):
    p, g, n = problem(M, N, K, act, 2)
    b32 = torch.randn(n, generator=g, device=DEV)
    check(p, keep=True)
    check(p, bias=b32.to(BF16), residual=values((M, N), g, False))
    if act != "swiglu":
        check(p, bias=b32, residual=torch.randn(M, N, generator=g, device=DEV), dtype=torch.float32, keep=True)
        check(p, bias=b32.to(BF16), dtype=torch.float32)
    check(p, bias=b32, keep=True)


@pytest.mark.parametrize("M,N,K,act", [(1, 256, 7168, "none"), (8, 2048, 7168, "swiglu"), (64, 4096, 2048, "gelu"),
                                       (2048, 256, 7168, "none"), (1000, 2056, 1000, "silu"), (4091, 520, 2048, "none"),
                                       (5000, 8, 1024, "none"), (300, 5000, 520, "relu")])
def test_larger_layers(M, N, K, act):
    p, g, n = problem(M, N, K, act, 3)
    check(p, bias=torch.randn(n, generator=g, device=DEV).to(BF16), residual=values((M, N), g, False), keep=act != "none")
    if act != "swiglu":
        check(p, dtype=torch.float32)


def test_values_far_from_zero():
    for act in ACTS:
        p, g, n = problem(20, 64, 64, act, 4)
        p["x"] = p["x"] * 30
        check(p, keep=True)


def test_residual_in_place_and_no_rows():
    p, g, n = problem(70, 264, 136, "relu", 5)
    r = values((70, 264), g, False)
    want = ep.linear(**p, residual=r)
    out = r.clone()
    assert ep.linear(**p, residual=out, out=out) is out and torch.equal(out, want)
    r1 = r[:3].clone()
    p["x"] = p["x"][:3].contiguous()
    assert torch.equal(ep.linear(**p, residual=r1, out=r1), ep.linear(**p, residual=r[:3].contiguous()))
    p["x"] = p["x"][:0]
    assert ep.linear(**p).shape == (0, 264)


def check_back(M, N, K, act, seed, dtype=torch.float32, add=False, exact=False):
    p, g, n = problem(M, N, K, act, seed, exact)
    dy = values((M, N), g, exact)
    z = None if act == "none" else (values((M, n), g, False) * 2)
    base = torch.randn(n, K, generator=g, device=DEV).to(dtype) if add else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dw = base.clone() if add else None
    grads = ep.linear_backward(dy, p["x"], p["w"], z, act, dw=dw, add=dw, dtype=dtype, status=status)
    assert ep.status_read(status) == 0 and (grads.dz is None) == (z is None)
    d, off = dy.double(), torch.zeros(M, N, device=DEV, dtype=torch.float64)
    if act == "swiglu":
        d, off = ref.gated_back(z.double(), d, off)
    elif z is not None:
        d, off = ref.activation_back(z.double(), d, act)
    # the sum of M values of fp32, each off by its own bound
    assert ref.close(grads.dbias, d.sum(0), ref.gamma(M) * (d.abs() + off).sum(0) + off.sum(0))
    if z is not None:
        assert ref.close(grads.dz, d, off)
        d = grads.dz
    assert ref.close(grads.dx, *ref.product(d, p["w"].T))
    want, off = ref.product(d.T, p["x"].T)
    if add:
        want = want + base.double()
        off = off + 2.0 ** -24 * (want.abs() + off)
    assert ref.close(grads.dw, want, off)
    return dy, p, z, grads


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 16, 8), (7, 48, 136), (65, 128, 264), (300, 400, 1000), (2000, 272, 520)])
def test_backward(act, M, N, K):
    check_back(M, N, K, act, 6)
    check_back(M, N, K, act, 7, BF16)
    check_back(M, N, K, act, 8, add=True)


@pytest.mark.parametrize("scale", [1.0, 1.0390625, -1.6171875])
def test_gelu_backward_keeps_its_digits_where_its_terms_cancel(scale):
    """The bias gradient of one row is the unrounded dy gelu'(z).  In parts of 2^-24:
    two roundings of the value; of dy v^3 the last step and the first coefficient
    of r (1/4 each, of a value below 1/2) and the smaller ones (1/8 in all); of dy
    the fit, 0.1."""
    bits = torch.arange(0x3000, 0x3F80, dtype=torch.int32)
    z = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(BF16).to(DEV).view(1, -1)
    x, w = torch.zeros(1, 8, dtype=BF16, device=DEV), torch.zeros(z.shape[1], 8, dtype=BF16, device=DEV)
    got = ep.linear_backward(torch.full_like(z, scale), x, w, z, "gelu").dbias.double()
    v = z[0].double()
    want = scale * (ref.cdf(v) + v * ref.phi(v))
    off = 2 * want.abs() + abs(scale) * (0.625 * v.abs() ** 3 + 0.1)
    assert want.abs().min() < 1e-3 * abs(scale)
    assert ((got - want).abs() <= 2.0 ** -24 * off).all()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_infinite_gradients_stay_infinite(act):
    z = torch.tensor([[-2.0, -0.9, -0.7, -0.5, -0.0117, 0.0117, 0.5, 0.75, 0.99, 2.0, 1.0, -1.0, 3.0, 0.125, -0.25, 4.0]],
                     dtype=BF16, device=DEV)
    x, w = torch.zeros(1, 8, dtype=BF16, device=DEV), torch.zeros(16, 8, dtype=BF16, device=DEV)
    v = z.double()
    slope = ref.activation_back(v, torch.ones_like(v), act)[0]
    for inf in (float("inf"), -float("inf")):
        got = ep.linear_backward(torch.full_like(z, inf), x, w, z, act, with_dx=False, with_dw=False).dz
        live = slope != 0
        assert torch.equal(got[live].double(), (slope * inf)[live])


@pytest.mark.parametrize("M,N,K", [(4000, 64, 512), (5271, 128, 264), (8192, 256, 1032), (9000, 8, 8)])
def test_weight_gradients_of_rows_in_parts(M, N, K):
    """Few tiles and many rows: the rows are summed in parts."""
    assert ep.linear_backward_workspace_bytes(M, K, N) > 0
    p, g, n = problem(M, N, K, "none", 15, exact=True)
    dy, base = values((M, N), g, True), values((N, K), g, True)
    want = ref.product(dy.T, p["x"].T)[0]
    for dtype in (torch.float32, BF16):
        got = ep.linear_backward(dy, p["x"], p["w"], dtype=dtype)
        assert torch.equal(got.dw, want.to(dtype)) and torch.equal(got.dbias, dy.double().sum(0).float())
        dw = base.to(dtype, copy=True)
        ep.linear_backward(dy, p["x"], p["w"], dw=dw, add=dw, with_dx=False)
        assert torch.equal(dw, (want + base.double()).to(dtype))
    check_back(M, N, K, "relu", 16)
    need = ep.linear_backward_workspace_bytes(M, K, N)
    for size, fits in ((need, True), (need - 1, False)):
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        if fits:
            assert torch.equal(ep.linear_backward(dy, p["x"], p["w"], workspace=ws).dw, want.float())
        else:
            with pytest.raises(ep.EpError):
                ep.linear_backward(dy, p["x"], p["w"], workspace=ws)
            ep.linear_backward(dy, p["x"], p["w"], workspace=ws, with_dw=False)


def test_backward_of_parts():
    dy, p, z, all_ = check_back(130, 64, 72, "silu", 9)
    for with_dx in (False, True):
        for with_dw in (False, True):
            for with_dbias in (False, True):
                got = ep.linear_backward(dy, p["x"], p["w"], z, "silu", with_dx=with_dx, with_dw=with_dw,
                                         with_dbias=with_dbias)
                assert torch.equal(got.dz, all_.dz)
                for name, w in (("dx", with_dx), ("dw", with_dw), ("dbias", with_dbias)):
                    v = getattr(got, name)
                    assert torch.equal(v, getattr(all_, name)) if w else v is None
    empty = ep.linear_backward(dy[:0], p["x"][:0], p["w"], z[:0], "silu")
    assert (empty.dw == 0).all() and (empty.dbias == 0).all() and empty.dx.shape == (0, 72)
    empty = ep.linear_backward(dy[:0], p["x"][:0], p["w"], dw=torch.ones(64, 72, device=DEV), add=torch.ones(64, 72, device=DEV))
    assert (empty.dw == 1).all() and (empty.dbias == 0).all()


def test_derivatives_far_from_zero():
    for act in ("relu", "silu", "gelu", "swiglu"):
        g = gen(10)
        n = 32 if act == "swiglu" else 16
        z = values((64, n), g, False) * 40
        dy = values((64, 16), g, False)
        got = ep.linear_backward(dy, values((64, 8), g, False), values((n, 8), g, False), z, act)
        d, off = (ref.gated_back(z.double(), dy.double(), torch.zeros_like(dy.double())) if act == "swiglu" else
                  ref.activation_back(z.double(), dy.double(), act))
        assert ref.close(got.dz, d, off), act


def test_graphs_share_no_state():
    """Two captured graphs of the same layer, replayed on two streams at once."""
    p, g, n = problem(40, 512, 2048, "gelu", 11)
    want = ep.linear(**p)
    graphs, outs, streams = [], [], []
    for _ in range(2):
        s, gr, out = torch.cuda.Stream(), torch.cuda.CUDAGraph(), full((40, 512))
        with torch.cuda.graph(gr, stream=s):
            for _ in range(5):
                ep.linear(**p, out=out)
        graphs.append(gr), outs.append(out), streams.append(s)
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_outputs_stay_inside_their_buffers():
    n = 4096
    for M in (1, 9, 37, 140):
        p, g, wide = problem(M, 136, 264, "silu", 12)
        for dt in (BF16, torch.float32):
            raw, rawz = full((2 * n + M * 136,), dt), full((2 * n + M * 136,))
            ep.linear(**p, out=raw[n:-n].view(M, 136), z=rawz[n:-n].view(M, 136))
            for r in (raw, rawz):
                assert (r[:n] == FREE).all() and (r[-n:] == FREE).all() and not (r[n:-n] == FREE).any()


def test_linear_refusals():
    p, g, n = problem(4, 64, 64, "none", 13)
    x, w, dy = p["x"], p["w"], values((4, 64), g, True)
    for bad in (dict(x=x.float()), dict(w=w.t().contiguous()[:, :8]), dict(activation="tanh"), dict(bias=w[:, :1]),
                dict(bias=torch.zeros(64, dtype=torch.float16, device=DEV)), dict(residual=x.float()),
                dict(dtype=torch.float16), dict(z=x.float()), dict(out=full((4, 32))), dict(x=x.cpu()),
                dict(activation="swiglu", dtype=torch.float32)):
        with pytest.raises(ValueError):
            ep.linear(**{**p, **bad})
    with pytest.raises(ep.EpError):
        ep.linear(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(ep.EpError):
        ep.linear(x, w[:48].contiguous(), activation="swiglu")   # 24 channels are no multiple of 16
    for bad in (dict(z=x), dict(dz=x), dict(activation="silu"), dict(dw=full((64, 64), torch.float16)),
                dict(with_dw=False, add=full((64, 64))), dict(dbias=full((64,)))):
        with pytest.raises(ValueError):
            ep.linear_backward(**{**dict(dy=dy, x=x, w=w), **bad})


# ---- the combine's gradient ---------------------------------------------------


@pytest.mark.parametrize("T,H,E,k", [(1, 8, 4, 1), (1, 2048, 128, 8), (3, 264, 8, 3), (200, 1000, 16, 4), (64, 7168, 64, 8),
                                     (130, 136, 40, 32), (1000, 64, 16, 12), (5000, 256, 64, 8), (17000, 64, 8, 2)])
@pytest.mark.parametrize("kind", ["contiguous", "masked"])
def test_combine_backward(T, H, E, k, kind):
    g = gen(T + H)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.int()
    idx[torch.rand(T, k, generator=g, device=DEV) < 0.1] = -1
    capacity = max(1, T * k // E) if kind == "masked" else 0   # some pairs overflow
    lay = ep.layout(idx, E, 1, kind, capacity)
    rows = E * capacity if kind == "masked" else T * k
    y, dout = values((rows, H), g, False), values((T, H), g, False)
    w = torch.randn(T, k, generator=g, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dy, dw = ep.combine_backward(dout, y, w, lay.dst_row, dy=full((rows, H)), dw=full((T, k), torch.float32), status=status)
    assert ep.status_read(status) == 0
    by_pair, want, off = ref.combine_back(dout, y, w, lay.dst_row)
    assert ref.close(dw, want, off)
    live = lay.dst_row >= 0
    # one fp32 product, rounded again to bf16
    assert ref.close(dy[lay.dst_row[live].long()], by_pair[live], 2.0 ** -24 * by_pair[live].abs() + 1e-40)
    free = torch.ones(rows, dtype=torch.bool, device=DEV)
    free[lay.dst_row[live].long()] = False
    assert (dy[free] == FREE).all() and (dw[~live] == 0).all()
    again = ep.combine_backward(dout, y, w, lay.dst_row, dy=full((rows, H)))
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)


def test_combine_backward_skips_and_reports_bad_rows():
    g = gen(20)
    y, dout, w = values((4, 16), g, False), values((2, 16), g, False), torch.ones(2, 3, device=DEV)
    dst = torch.tensor([[0, 4, -2], [-1, 3, 1 << 30]], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dy, dw = ep.combine_backward(dout, y, w, dst, dy=full((4, 16)), status=status)
    assert ep.status_read(status) == ep.EP_FLAG_BAD_ROW
    assert torch.equal(dy[0], dout[0]) and torch.equal(dy[3], dout[1]) and (dy[1:3] == FREE).all()
    assert torch.equal(dw == 0, torch.tensor([[False, True, True], [True, False, True]], device=DEV))


def test_combine_backward_refusals_and_no_tokens():
    g = gen(21)
    y, dout, w = values((4, 16), g, False), values((2, 16), g, False), torch.ones(2, 2, device=DEV)
    dst = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    for bad in (dict(y=y.float()), dict(dout=dout[:, :8].contiguous()), dict(topk_w=w[:1]), dict(dst_row=dst.long()),
                dict(dy=full((3, 16))), dict(dw=full((2, 2)))):
        with pytest.raises(ValueError):
            ep.combine_backward(**{**dict(dout=dout, y=y, topk_w=w, dst_row=dst), **bad})
    dy, dw = ep.combine_backward(dout[:0], y, w[:0], dst[:0], dy=full((4, 16)))
    assert (dy == FREE).all() and dw.shape == (0, 2)
