"""The experts' BF16 products and their gradients against plain 64-bit
definitions: bit-equal on data whose every fp32 step is exact, within the
derived error bounds on random data."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import moe_reference as moe
import product_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
FREE = -77.0  # what rows of no expert hold before and after


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def values(shape, g, exact):
    """Normal values, or ones whose products and sums are exact in fp32."""
    if exact:
        return (torch.randint(-4, 5, shape, generator=g, device=DEV) * 0.5).to(BF16)
    return torch.randn(shape, generator=g, device=DEV).to(BF16)


class Problem:
    """Segments of `counts` rows, `gap` rows of no expert after each contiguous
    one.  Rows of no expert hold NaN in every buffer."""

    def __init__(self, counts, kind, seed, exact=False, capacity=None, gap=0):
        self.g, self.exact, self.counts, self.kind = gen(seed), exact, counts, kind
        E = len(counts)
        if kind == "masked":
            self.capacity = max(counts) if capacity is None else capacity
            first = [e * self.capacity for e in range(E)]
            self.rows = E * self.capacity
        else:
            self.capacity, first, at = 0, [], 0
            for n in counts:
                first.append(at)
                at += n + gap
            self.rows = at
        self.cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.off = torch.tensor(first + [self.rows], dtype=torch.int32, device=DEV)
        self.segments = moe.segments(self.cnt, self.off, kind, self.capacity, self.rows)
        self.at = (self.cnt, self.off, kind, self.capacity)

    def buffer(self, width):
        b = torch.full((self.rows, width), float("nan"), dtype=BF16, device=DEV)
        for _, a, z in self.segments:
            b[a:z] = values((z - a, width), self.g, self.exact)
        return b

    def weights(self, *shape):
        w = values((len(self.counts),) + shape, self.g, self.exact)
        return w if self.exact else (w.float() * shape[-1] ** -0.5).to(BF16)

    def free_rows_kept(self, out):
        free = torch.ones(self.rows, dtype=torch.bool, device=DEV)
        for _, a, z in self.segments:
            free[a:z] = False
        return (out[free] == FREE).all()


def full(shape, dtype=BF16):
    return torch.full(shape, FREE, dtype=dtype, device=DEV)


def same(got, want, off, exact):
    return torch.equal(got, want.to(got.dtype)) if exact else ref.close(got, want, off)


def check_forward(p, N, K):
    x, w, status = p.buffer(K), p.weights(N, K), torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ep.group_gemm(x, w, *p.at, out=full((p.rows, N)), status=status)
    assert ep.status_read(status) == 0 and p.free_rows_kept(out)
    for e, a, z in p.segments:
        assert same(out[a:z], *ref.product(x[a:z], w[e]), p.exact), (e, a, z)
    again = ep.group_gemm(x, w, *p.at, out=full((p.rows, N)))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the order of every sum is fixed


def check_dgrad(p, N, K):
    dy, w, status = p.buffer(N), p.weights(N, K), torch.zeros(1, dtype=torch.int32, device=DEV)
    dx = ep.group_gemm_dgrad(dy, w, *p.at, dx=full((p.rows, K)), status=status)
    assert ep.status_read(status) == 0 and p.free_rows_kept(dx)
    for e, a, z in p.segments:
        assert same(dx[a:z], *ref.product(dy[a:z], w[e].T), p.exact), (e, a, z)


def check_wgrad(p, N, K, dtype=torch.float32, add=False):
    dy, x, status = p.buffer(N), p.buffer(K), torch.zeros(1, dtype=torch.int32, device=DEV)
    base = values((len(p.counts), N, K), p.g, p.exact).to(dtype) if add else None
    dw = base.clone() if add else full((len(p.counts), N, K), dtype)
    ep.group_gemm_wgrad(dy, x, *p.at, dw=dw, add=dw if add else None, status=status)
    assert ep.status_read(status) == 0
    segs = {e: (a, z) for e, a, z in p.segments}
    for e in range(len(p.counts)):
        a, z = segs.get(e, (0, 0))
        want, off = ref.product(dy[a:z].T, x[a:z].T)
        if add:
            want = want + base[e].double()
            off = off + 2.0 ** -24 * (want.abs() + off)
        assert same(dw[e], want, off, p.exact), e


def check_swiglu(p, I, K):
    x, w, status = p.buffer(K), p.weights(2 * I, K), torch.zeros(1, dtype=torch.int32, device=DEV)
    z = full((p.rows, 2 * I))
    out = ep.group_gemm_swiglu(x, w, *p.at, out=full((p.rows, I)), z=z, status=status)
    assert ep.status_read(status) == 0 and p.free_rows_kept(out) and p.free_rows_kept(z)
    for e, a, b in p.segments:
        y, dy = ref.product(x[a:b], w[e])
        assert same(z[a:b], y, dy, p.exact), (e, a, b)
        assert ref.close(out[a:b], *ref.gated(y, dy)), (e, a, b)
    assert torch.equal(out, ep.group_gemm_swiglu(x, w, *p.at, out=full((p.rows, I))))  # without z


def check_swiglu_dgrad(p, H, I):
    dy, w, z, status = p.buffer(H), p.weights(H, I), p.buffer(2 * I), torch.zeros(1, dtype=torch.int32, device=DEV)
    dz = ep.group_gemm_swiglu_dgrad(dy, w, z, *p.at, dz=full((p.rows, 2 * I)), status=status)
    assert ep.status_read(status) == 0 and p.free_rows_kept(dz)
    for e, a, b in p.segments:
        dh, ddh = ref.product(dy[a:b], w[e].T)
        assert ref.close(dz[a:b], *ref.gated_back(z[a:b].double(), dh, ddh)), (e, a, b)


COUNTS = [[1], [0, 1, 0], [7, 0, 130, 64], [127, 128, 129], [300, 1, 0, 33, 5], [0, 0, 0], [16, 8, 24, 32, 40, 48, 2],
          [257, 383, 64, 255, 256], [15, 17, 31, 63, 65, 95, 97]]
WIDTHS = [(128, 128), (8, 8), (8, 256), (264, 384), (1000, 1024), (136, 640), (520, 72)]


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", WIDTHS)
def test_products_are_exact_on_exact_data(counts, kind, N, K):
    p = Problem(counts, kind, 1, exact=True, gap=3)
    check_forward(p, N, K)
    check_dgrad(p, N, K)
    check_wgrad(p, N, K)
    check_wgrad(p, N, K, BF16)


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("I,K", [(16, 8), (48, 136), (128, 128), (400, 1000), (144, 2056)])
def test_gated_products(counts, kind, I, K):
    p = Problem(counts, kind, 2, gap=2)
    check_swiglu(p, I, K)
    check_swiglu_dgrad(p, K, I)


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts,N,K", [([64] * 16, 256, 7168), ([5, 0, 200, 1], 520, 2048), ([1], 5000, 7168),
                                        ([700, 20], 2056, 128), ([3] * 60, 896, 384), ([2000, 100], 776, 1032)])
def test_products_within_bounds(counts, kind, N, K):
    p = Problem(counts, kind, 3)
    check_forward(p, N, K)
    check_dgrad(p, N, K)
    check_wgrad(p, N, K)
    check_wgrad(p, N, K, BF16, add=True)


def test_many_experts_and_many_tiles():
    check_forward(Problem([3, 0, 1] * 300, "contiguous", 4, exact=True), 136, 72)
    check_wgrad(Problem([3, 0, 1] * 100, "contiguous", 4, exact=True), 136, 72)
    p = Problem([1500, 3000, 700], "contiguous", 5, exact=True)
    check_forward(p, 2048, 64)
    check_dgrad(p, 64, 2048)
    check_wgrad(p, 1032, 1032)


def test_sums_that_are_added_in_parts():
    # fp32 sums are cut every 512 rows: whole parts, one row more, 16 more, and a short last one
    p = Problem([512, 513, 1024, 1040, 511, 4097], "contiguous", 18, exact=True, gap=1)
    check_wgrad(p, 136, 200)
    check_wgrad(p, 64, 328, add=True)
    check_wgrad(p, 136, 200, BF16)


def test_weight_gradients_are_added():
    p = Problem([70, 0, 3], "contiguous", 6, exact=True)
    check_wgrad(p, 264, 136, torch.float32, add=True)
    check_wgrad(p, 264, 136, BF16, add=True)
    dy, x, base = p.buffer(8), p.buffer(8), torch.ones(3, 8, 8, device=DEV)
    dw = ep.group_gemm_wgrad(dy, x, *p.at, add=base)
    assert torch.equal(dw, ep.group_gemm_wgrad(dy, x, *p.at) + 1) and (base == 1).all()


def test_gates_far_from_zero():
    p = Problem([40], "contiguous", 7)
    dy, w, z = p.buffer(64), p.weights(64, 32), 60 * p.buffer(64)
    dz = ep.group_gemm_swiglu_dgrad(dy, w, z, *p.at)
    assert ref.close(dz, *ref.gated_back(z.double(), *ref.product(dy, w[0].T)))
    x, w13 = 100 * p.buffer(64), p.weights(64, 64)
    y, off = ref.product(x, w13[0])
    assert ref.close(ep.group_gemm_swiglu(x, w13, *p.at), *ref.gated(y, off))


def test_overflowing_counts_and_segments_outside_the_buffer():
    p = Problem([3, 130, 64, 0], "masked", 8, exact=True, capacity=64)  # 130 > capacity
    check_forward(p, 144, 256)
    check_dgrad(p, 144, 256)
    check_wgrad(p, 144, 256)
    p = Problem([10, 20, 30], "contiguous", 9, exact=True)
    x, dy, w = p.buffer(128), p.buffer(64), p.weights(64, 128)
    p.cnt[2] = 90000           # reaches past the buffer
    p.cnt[0] = -4
    p.off[1] = -2
    for call in (lambda s: ep.group_gemm(x, w, *p.at, out=full((60, 64)), status=s),
                 lambda s: ep.group_gemm_dgrad(dy, w, *p.at, dx=full((60, 128)), status=s),
                 lambda s: ep.group_gemm_wgrad(dy, x, *p.at, status=s)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = call(status)
        assert ep.status_read(status) == ep.EP_FLAG_BAD_ROW
        if out.dim() == 2:
            want = ref.product(x[30:], w[2])[0] if out.shape[1] == 64 else ref.product(dy[30:], w[2].T)[0]
            assert torch.equal(out[30:], want.to(BF16)) and (out[:30] == FREE).all()
        else:
            assert (out[:2] == 0).all() and torch.equal(out[2], ref.product(dy[30:].T, x[30:].T)[0].float())


def test_no_rows():
    cnt, off = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    x, w = torch.zeros(0, 64, dtype=BF16, device=DEV), torch.zeros(2, 64, 64, dtype=BF16, device=DEV)
    assert ep.group_gemm(x, w, cnt, off).shape == (0, 64) and ep.group_gemm_dgrad(x, w, cnt, off).shape == (0, 64)
    assert (ep.group_gemm_wgrad(x, x, cnt, off, dw=full((2, 64, 64), torch.float32)) == 0).all()


def test_outputs_stay_inside_their_buffers():
    p = Problem([37, 100], "contiguous", 10)
    x, dy, w13, w2, z = p.buffer(264), p.buffer(264), p.weights(96, 264), p.weights(264, 48), p.buffer(96)
    n = 4096

    def guarded(shape, dtype=BF16):
        raw = torch.full((2 * n + shape.numel(),), FREE, dtype=dtype, device=DEV)
        return raw, raw[n:-n].view(shape)

    S = torch.Size
    for call, shapes in ((lambda o, zz: ep.group_gemm_swiglu(x, w13, *p.at, out=o, z=zz), (S((137, 48)), S((137, 96)))),
                         (lambda o: ep.group_gemm(x, w13, *p.at, out=o), (S((137, 96)),)),
                         (lambda o: ep.group_gemm_dgrad(dy, w2, *p.at, dx=o), (S((137, 48)),)),
                         (lambda o: ep.group_gemm_swiglu_dgrad(dy, w2, z, *p.at, dz=o), (S((137, 96)),)),
                         (lambda o: ep.group_gemm_wgrad(dy, z, *p.at, dw=o), (S((2, 264, 96)),))):
        bufs = [guarded(s, torch.float32 if len(s) == 3 else BF16) for s in shapes]
        call(*(v for _, v in bufs))
        for raw, v in bufs:
            assert (raw[:n] == FREE).all() and (raw[-n:] == FREE).all() and torch.isfinite(v.float()).all()


def test_buffers_on_16_but_not_32_bytes():
    p = Problem([37, 100], "contiguous", 11, exact=True)
    x, dy, w = p.buffer(64), p.buffer(96), p.weights(96, 64)

    def off(shape, dtype=BF16):
        n = shape[0] * shape[1] * (shape[2] if len(shape) == 3 else 1)
        skip = 8 if dtype is BF16 else 4
        t = torch.zeros(n + 64, dtype=dtype, device=DEV)[skip:skip + n].view(shape)
        assert t.data_ptr() % 32 == 16
        return t

    x2, dy2, w2 = off(x.shape).copy_(x), off(dy.shape).copy_(dy), off(w.shape).copy_(w)
    assert torch.equal(ep.group_gemm(x2, w2, *p.at, out=off((137, 96))), ep.group_gemm(x, w, *p.at))
    assert torch.equal(ep.group_gemm_dgrad(dy2, w2, *p.at, dx=off((137, 64))), ep.group_gemm_dgrad(dy, w, *p.at))
    for dt in (torch.float32, BF16):
        assert torch.equal(ep.group_gemm_wgrad(dy2, x2, *p.at, dw=off((2, 96, 64), dt)),
                           ep.group_gemm_wgrad(dy, x, *p.at, dtype=dt))


def test_nan_and_infinity_stay_in_their_row_and_channel():
    p = Problem([130, 20], "contiguous", 12, exact=True)
    x, dy, w = p.buffer(256), p.buffer(264), p.weights(264, 256)
    x[5, 200] = float("inf")
    w[1, 17, 3] = float("nan")
    dy[140, 9] = float("nan")
    bad = ~torch.isfinite(ep.group_gemm(x, w, *p.at).float())
    want = torch.zeros_like(bad)
    want[5] = w[0, :, 200] != 0      # and NaN where the weight is 0
    want[5] |= w[0, :, 200] == 0
    want[130:, 17] = True
    assert torch.equal(bad, want)
    bad = ~torch.isfinite(ep.group_gemm_dgrad(dy, w, *p.at).float())
    want = torch.zeros_like(bad)
    want[130:, 3] = True
    want[140] = True
    assert torch.equal(bad, want)
    bad = ~torch.isfinite(ep.group_gemm_wgrad(dy, x, *p.at))
    want = torch.zeros_like(bad)
    want[0, :, 200] = True
    want[1, 9] = True
    assert torch.equal(bad, want)


def test_rows_beyond_32_bit_offsets():
    # 3 * 2^20 rows of 1,024 channels: byte offsets of the last expert pass 2^32
    K, N, cap = 1024, 64, 1 << 20
    p = Problem([1, 3, 150], "masked", 13, exact=True, capacity=cap)
    check_forward(p, N, K)
    check_dgrad(p, N, K)
    check_wgrad(p, N, K)


def test_graph_capture_and_another_stream():
    p = Problem([65, 0, 7], "contiguous", 14, exact=True)
    x, dy, w, z = p.buffer(64), p.buffer(96), p.weights(96, 64), p.buffer(96)
    out, dx, dw = full((72, 96)), full((72, 64)), full((3, 96, 64), torch.float32)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.group_gemm(x, w, *p.at, out=out)
        ep.group_gemm_dgrad(dy, w, *p.at, dx=dx)
        ep.group_gemm_wgrad(dy, x, *p.at, dw=dw)
    x.copy_(values(x.shape, p.g, True))
    dy.copy_(values(dy.shape, p.g, True))
    p.cnt.copy_(torch.tensor([0, 60, 7], dtype=torch.int32, device=DEV))
    p.off.copy_(torch.tensor([0, 5, 65, 72], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[5:65], ref.product(x[5:65], w[1])[0].to(BF16)) and (out[:5] == FREE).all()
    assert torch.equal(dx[65:], ref.product(dy[65:], w[2].T)[0].to(BF16))
    assert (dw[0] == 0).all() and torch.equal(dw[1], ref.product(dy[5:65].T, x[5:65].T)[0].float())


def test_calls_on_two_streams_at_once():
    ps = [Problem([300, 5, 64], "contiguous", 15 + i, exact=True) for i in range(2)]
    data = [(p.buffer(256), p.weights(512, 256)) for p in ps]
    want = [ep.group_gemm(x, w, *p.at, out=full((p.rows, 512))) for p, (x, w) in zip(ps, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(50):
        for i, (p, (x, w), s) in enumerate(zip(ps, data, streams)):
            with torch.cuda.stream(s):
                got[i].append(ep.group_gemm(x, w, *p.at))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)


def test_refusals():
    p = Problem([4, 4], "contiguous", 17)
    x, dy, w, z = p.buffer(64), p.buffer(96), p.weights(96, 64), p.buffer(128)
    good = dict(x=x, w=w, expert_counts=p.cnt, expert_offsets=p.off)
    for name, bad in (("x", x.float()), ("x", x.t()), ("x", x.cpu()), ("x", x[:, :56].contiguous()), ("w", w.half()),
                      ("w", w[0]), ("expert_counts", p.cnt.long()), ("expert_counts", p.cnt[:1]), ("kind", "other"),
                      ("out", full((8, 64))), ("out", full((8, 96), torch.float32)),
                      ("status", torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            ep.group_gemm(**{**good, name: bad})
    for call in (lambda: ep.group_gemm_dgrad(x, w, *p.at), lambda: ep.group_gemm_swiglu_dgrad(dy, w, dy, *p.at),
                 lambda: ep.group_gemm_swiglu(x, w, *p.at, z=x), lambda: ep.group_gemm_wgrad(dy, x[:4].contiguous(), *p.at),
                 lambda: ep.group_gemm_wgrad(dy, x, *p.at, dtype=torch.float16),
                 lambda: ep.group_gemm_wgrad(dy, x, *p.at, dw=full((2, 64, 96))),
                 lambda: ep.group_gemm_wgrad(dy, x, *p.at, add=full((2, 96, 64)))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ep.EpError):
        ep.group_gemm(x, w, p.cnt, None, "masked", 100)        # rows < E * capacity
    with pytest.raises(ep.EpError):
        ep.group_gemm(x, w, p.cnt, None)                       # contiguous needs offsets
    with pytest.raises(ep.EpError):                            # 24 gate rows are no multiple of 16
        ep.group_gemm_swiglu(x, w[:, :48].contiguous(), *p.at)
