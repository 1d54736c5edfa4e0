"""The experts' FP8 products (ep_group_gemm_fp8, ep_group_gemm_swiglu_fp8)
against plain 64-bit definitions: bit-equal on data whose every fp32 step is
exact, within the derived error bounds on random data."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import moe_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def random_codes(shape, g):
    return (100.0 * torch.randn(shape, generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def small_codes(shape, g):
    """Codes of -2, -1, -0.5, 0, 0.5, 1, 2: sums of their products stay exact in fp32."""
    v = torch.tensor([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 2.0], device=DEV)
    return v[torch.randint(0, 7, shape, generator=g, device=DEV)].to(torch.float8_e4m3fn).view(torch.uint8)


def powers(shape, g):
    return torch.ldexp(torch.ones(shape, device=DEV), torch.randint(-2, 2, shape, generator=g, device=DEV).int())


def problem(counts, kind, K, N, seed, exact=False, capacity=None, gap=0):
    """Buffers of `counts` rows per expert; `gap` rows of no expert after each
    contiguous segment.  Rows of no expert hold NaN codes and scales."""
    g = gen(seed)
    E = len(counts)
    if kind == "masked":
        capacity = max(counts) if capacity is None else capacity
        first = [e * capacity for e in range(E)]
        rows = E * capacity
    else:
        first, at = [], 0
        for n in counts:
            first.append(at)
            at += n + gap
        rows = at
        capacity = 0
    codes, scales = (small_codes, powers) if exact else (
        random_codes, lambda s, g: (0.75 + 0.5 * torch.rand(s, generator=g, device=DEV)) / 100)
    a_q = torch.full((rows, K), 0x7F, dtype=torch.uint8, device=DEV)
    a_s = torch.full((rows, K // 128), float("nan"), device=DEV)
    for n, f in zip(counts, first):
        n = min(n, capacity) if kind == "masked" else n
        a_q[f:f + n] = codes((n, K), g)
        a_s[f:f + n] = scales((n, K // 128), g)
    w_q, w_s = codes((E, N, K), g), scales((E, (N + 127) // 128, K // 128), g)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    off = torch.tensor(first + [rows], dtype=torch.int32, device=DEV)
    return dict(a_q=a_q, a_scale=a_s, w_q=w_q, w_scale=w_s, expert_counts=cnt, expert_offsets=off, kind=kind,
                capacity=capacity), rows


def check_plain(p, rows, exact=False):
    N = p["w_q"].shape[1]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device=DEV)
    ep.group_gemm_fp8(**p, out=out, status=status)
    assert ep.status_read(status) == 0
    again = ep.group_gemm_fp8(**p, out=torch.full_like(out, -77.0))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the order of every sum is fixed
    free = torch.ones(rows, dtype=torch.bool, device=DEV)
    for e, a, b in ref.segments(p["expert_counts"], p["expert_offsets"], p["kind"], p["capacity"], rows):
        y, dy = ref.product(p["a_q"], p["a_scale"], p["w_q"], p["w_scale"], a, b, e)
        if exact:
            assert torch.equal(out[a:b], y.to(torch.float32).to(torch.bfloat16)), (e, a, b)
        else:
            assert ((out[a:b].double() - y).abs() <= 2.0 ** -8 * (y.abs() + dy) + dy).all(), (e, a, b)
        free[a:b] = False
    assert (out[free] == -77.0).all()


def check_swiglu(p, rows):
    I = p["w_q"].shape[1] // 2
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.full((rows, I), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, I // 128), -77.0, device=DEV)
    ep.group_gemm_swiglu_fp8(**p, out_q=q, out_scale=s, status=status)
    assert ep.status_read(status) == 0
    free = torch.ones(rows, dtype=torch.bool, device=DEV)
    for e, a, b in ref.segments(p["expert_counts"], p["expert_offsets"], p["kind"], p["capacity"], rows):
        y, dy = ref.product(p["a_q"], p["a_scale"], p["w_q"], p["w_scale"], a, b, e)
        h, dh = ref.silu_mul(y[:, :I], y[:, I:], dy[:, :I], dy[:, I:])
        want, slack, sc, dsc = ref.flip_slack(h, dh)
        assert ((s[a:b].double() - sc).abs() <= dsc).all(), (e, a, b)
        assert ((ref.rows64(q[a:b], s[a:b]) - want).abs() <= slack * (1 + 2.0 ** -20)).all(), (e, a, b)
        free[a:b] = False
    assert (q[free] == 0x55).all() and (s[free] == -77.0).all()


COUNTS = [[1], [0, 1, 0], [7, 0, 130, 64], [127, 128, 129], [300, 1, 0, 33, 5], [0, 0, 0], [16, 8, 24, 32, 40, 48, 2],
          [257, 383, 64]]


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(128, 128), (256, 8), (384, 264), (1024, 1000), (640, 136)])
def test_product_is_exact_on_exact_data(counts, kind, K, N):
    p, rows = problem(counts, kind, K, N, 1, exact=True)
    check_plain(p, rows, exact=True)


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts,K,N", [([64] * 16, 7168, 256), ([5, 0, 200, 1], 2048, 520), ([1], 7168, 5000),
                                        ([700, 20], 128, 2056), ([3] * 60, 384, 896)])
def test_product_within_bounds(counts, kind, K, N):
    p, rows = problem(counts, kind, K, N, 2)
    check_plain(p, rows)


@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,I", [(128, 128), (384, 384), (1024, 256)])
def test_swiglu_within_bounds(counts, kind, K, I):
    p, rows = problem(counts, kind, K, 2 * I, 3)
    check_swiglu(p, rows)


@pytest.mark.parametrize("counts,K,I", [([64] * 8, 7168, 2048), ([1], 7168, 256), ([600], 2048, 1024)])
def test_swiglu_large(counts, K, I):
    p, rows = problem(counts, "contiguous", K, 2 * I, 4)
    check_swiglu(p, rows)


def test_swiglu_of_extreme_gates():
    # gates far below and above zero, and rows of zeros: exp overflows to the
    # limit 0, the scale falls back to the smallest block's
    p, rows = problem([40], "contiguous", 128, 256, 5)
    p["w_scale"].fill_(30.0)
    p["a_q"][3] = 0
    check_swiglu(p, rows)


def test_segments_with_gaps_and_overflowing_counts():
    p, rows = problem([3, 130, 0, 65], "contiguous", 256, 144, 6, exact=True, gap=5)
    check_plain(p, rows, exact=True)
    p, rows = problem([3, 130, 64, 0], "masked", 256, 144, 7, exact=True, capacity=64)  # 130 > capacity
    check_plain(p, rows, exact=True)


def test_segments_outside_the_buffer_are_cut_and_reported():
    p, rows = problem([10, 20, 30], "contiguous", 128, 128, 8, exact=True)
    p["expert_counts"][2] = 90000          # reaches past the buffer
    p["expert_counts"][0] = -4
    p["expert_offsets"][1] = -2
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((rows, 128), -77.0, dtype=torch.bfloat16, device=DEV)
    ep.group_gemm_fp8(**p, out=out, status=status)
    assert ep.status_read(status) == ep.EP_FLAG_BAD_ROW
    y, _ = ref.product(p["a_q"], p["a_scale"], p["w_q"], p["w_scale"], 30, 60, 2)
    assert torch.equal(out[30:], y.float().to(torch.bfloat16)) and (out[:30] == -77.0).all()


def test_outputs_stay_inside_their_buffers():
    p, rows = problem([37, 100], "contiguous", 256, 384 * 2, 9)
    I = 384
    raw = torch.full((4096 + rows * I + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    raws = torch.full((1024 + rows * 3 + 1024,), -7.0, device=DEV)
    ep.group_gemm_swiglu_fp8(**p, out_q=raw[4096:-4096].view(rows, I), out_scale=raws[1024:-1024].view(rows, 3))
    rawo = torch.full((2048 + rows * 2 * I + 2048,), -7.0, dtype=torch.bfloat16, device=DEV)
    ep.group_gemm_fp8(**p, out=rawo[2048:-2048].view(rows, 2 * I))
    torch.cuda.synchronize()
    assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()
    assert (raws[:1024] == -7).all() and (raws[-1024:] == -7).all()
    assert (rawo[:2048] == -7).all() and (rawo[-2048:] == -7).all()


def test_outputs_on_16_but_not_32_bytes():
    p, rows = problem([37, 100], "contiguous", 256, 512, 16, exact=True)
    raw = torch.zeros(rows * 512 + 64, dtype=torch.bfloat16, device=DEV)
    off = raw[8:8 + rows * 512].view(rows, 512)
    assert off.data_ptr() % 32 == 16
    assert torch.equal(ep.group_gemm_fp8(**p, out=off), ep.group_gemm_fp8(**p))
    want, scale = ep.group_gemm_swiglu_fp8(**p)
    rawq = torch.zeros(rows * 256 + 64, dtype=torch.uint8, device=DEV)
    q, s = ep.group_gemm_swiglu_fp8(**p, out_q=rawq[16:16 + rows * 256].view(rows, 256))
    assert torch.equal(q, want) and torch.equal(s, scale)


def test_nan_codes_stay_in_their_row():
    p, rows = problem([130, 20], "contiguous", 256, 264, 10, exact=True)
    p["a_q"][5, 200] = 0x7F
    p["w_q"][1, 17, 3] = 0xFF
    out = ep.group_gemm_fp8(**p).float()
    want = torch.zeros(rows, 264, dtype=torch.bool, device=DEV)
    want[5] = True
    want[130:, 17] = True
    assert torch.equal(torch.isnan(out), want)


def test_rows_beyond_32_bit_offsets():
    # 2^21 rows of 2,048 channels: byte offsets of the last expert pass 2^32
    K, N, cap = 2048, 256, 1 << 20
    g = gen(11)
    a_q = torch.zeros(3 * cap, K, dtype=torch.uint8, device=DEV)
    a_s = torch.ones(3 * cap, K // 128, device=DEV)
    cnt = torch.tensor([1, 3, 150], dtype=torch.int32, device=DEV)
    for e, n in enumerate([1, 3, 150]):
        a_q[e * cap:e * cap + n] = small_codes((n, K), g)
    p = dict(a_q=a_q, a_scale=a_s, w_q=small_codes((3, N, K), g), w_scale=powers((3, 2, 16), g), expert_counts=cnt,
             expert_offsets=None, kind="masked", capacity=cap)
    out = ep.group_gemm_fp8(**p)
    for e, n in enumerate([1, 3, 150]):
        y, _ = ref.product(a_q, a_s, p["w_q"], p["w_scale"], e * cap, e * cap + n, e)
        assert torch.equal(out[e * cap:e * cap + n], y.float().to(torch.bfloat16))


def test_dispatch_to_combine_through_the_products():
    """route -> layout_dispatch (FP8) -> both products -> combine, contiguous,
    aligned and masked layouts: the same result bit for bit."""
    T, H, I, E, k = 200, 512, 256, 16, 4
    g = gen(12)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    idx, w = ep.route(torch.randn(T, E, generator=g, device=DEV), k)
    w13, s13 = random_codes((E, 2 * I, H), g), torch.full((E, 2 * I // 128, H // 128), 4e-4, device=DEV)
    w2, s2 = random_codes((E, H, I), g), torch.full((E, H // 128, I // 128), 6e-4, device=DEV)
    outs = []
    for kind, capacity, align in (("contiguous", 0, 1), ("contiguous", 0, 64), ("masked", T, 1)):
        lay = ep.layout(idx, E, 1, kind, capacity, alignment=align)
        rows = E * capacity if kind == "masked" else T * k + E * (align - 1)
        q, s = ep.dispatch_fp8(x, lay.dst_row, rows, status=lay.status)
        hq, hs = ep.group_gemm_swiglu_fp8(q, s, w13, s13, lay.expert_counts, lay.expert_offsets, kind, capacity,
                                          status=lay.status)
        y = ep.group_gemm_fp8(hq, hs, w2, s2, lay.expert_counts, lay.expert_offsets, kind, capacity,
                              status=lay.status)
        outs.append(ep.combine(y, w, lay.dst_row, status=lay.status))
        assert ep.status_read(lay.status) == 0
    assert torch.isfinite(outs[0].float()).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_graph_capture_and_another_stream():
    p, rows = problem([65, 0, 7], "contiguous", 256, 256, 13, exact=True)
    out = torch.zeros(rows, 256, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.group_gemm_fp8(**p, out=out)
    p["a_q"].copy_(small_codes(p["a_q"].shape, gen(14)))
    g.replay()
    torch.cuda.synchronize()
    for e, a, b in ref.segments(p["expert_counts"], p["expert_offsets"], "contiguous", 0, rows):
        y, _ = ref.product(p["a_q"], p["a_scale"], p["w_q"], p["w_scale"], a, b, e)
        assert torch.equal(out[a:b], y.float().to(torch.bfloat16))


def test_refusals():
    p, rows = problem([4, 4], "contiguous", 256, 128, 15)
    for name, bad in (("a_q", p["a_q"].float()), ("a_scale", p["a_scale"][:, :1].contiguous()),
                      ("w_q", p["w_q"][:, :, :128].contiguous()), ("w_scale", p["w_scale"].half()),
                      ("expert_counts", p["expert_counts"].long()), ("expert_counts", p["expert_counts"][:1]),
                      ("kind", "other"), ("a_q", p["a_q"].t()), ("a_q", p["a_q"].cpu())):
        with pytest.raises(ValueError):
            ep.group_gemm_fp8(**{**p, name: bad})
    with pytest.raises(ValueError):
        ep.group_gemm_fp8(**p, out=torch.zeros(rows, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ep.EpError):
        ep.group_gemm_fp8(**{**p, "kind": "masked", "capacity": 100})   # rows < E * capacity
    with pytest.raises(ep.EpError):                                    # half of 128 rows is no whole block
        ep.group_gemm_swiglu_fp8(**p)
