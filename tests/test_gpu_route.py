"""The router's choice (ep_route) against a plain 64-bit definition: ids equal
everywhere, weights within the fp32 error of the formula."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import moe_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def check(logits, k, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    idx, w = ep.route(logits, k, status=status, **kw)
    rkw = {a: b for a, b in kw.items() if a not in ("topk_idx", "topk_w")}
    ri, rw = ref.route(logits, k, **rkw)
    assert torch.equal(idx.cpu().long(), ri)
    # exp of d = l - m: d is rounded once (|d| u), expf is good to 2 ulp; the
    # sum of at most E terms, the quotient and the scale add E + 8 roundings.
    # |d| <= 100 wherever the result is above the subnormals (1e-37).
    bound = (100 + logits.shape[1] + 16) * 2 * ref.U * rw.abs() + 1e-36
    assert ((w.cpu().double() - rw).abs() <= bound).all()
    return ep.status_read(status)


def logits_of(T, E, dtype, seed=0, spread=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g, device=DEV)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (3, 1, 1), (5, 31, 4), (33, 32, 32), (64, 33, 3), (129, 64, 6),
                                   (200, 65, 2), (257, 128, 8), (65, 255, 9), (31, 256, 32), (40, 257, 8),
                                   (17, 512, 16), (19, 513, 8), (9, 1000, 8), (7, 1024, 32)])
@pytest.mark.parametrize("scoring,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                                 ("sigmoid", False)])
def test_route_matches_the_definition(T, E, k, dtype, scoring, renormalize):
    # bf16 logits of 256 and more experts hold many equal values: ties by id
    assert check(logits_of(T, E, dtype, T + E), k, scoring=scoring, renormalize=renormalize, scale=2.5) == 0


@pytest.mark.parametrize("E,groups,keep,k", [(256, 8, 4, 8), (256, 8, 1, 8), (128, 4, 3, 6), (61 * 8, 8, 3, 8),
                                             (24, 8, 2, 6), (32, 32, 5, 5), (96, 32, 31, 32), (1024, 32, 4, 8),
                                             (100, 4, 4, 8), (26, 2, 1, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_limited_to_groups(E, groups, keep, k, dtype):
    g = torch.Generator(device=DEV).manual_seed(3)
    bias = 0.3 * torch.randn(E, generator=g, device=DEV)
    for b in (None, bias):
        assert check(logits_of(120, E, dtype, E), k, bias=b, groups=groups, groups_per_token=keep) == 0


def test_route_ties_signed_zeros_and_whole_rows_equal():
    l = torch.zeros(6, 40, device=DEV)
    l[1] = -0.0
    l[2, ::2] = -0.0                        # -0 and +0 are one key
    l[3] = 1.5
    l[4, 7] = l[4, 33] = l[4, 12] = 2.0
    l[5] = -3.0e38
    check(l, 5)
    check(l, 5, groups=4, groups_per_token=2)


def test_route_masks_infinities_and_nan():
    l = logits_of(12, 70, torch.float32, 5)
    l[0] = -INF                             # nothing left: ids -1, weights 0
    l[1, 3:] = -INF                         # fewer than k left
    l[2, 10] = INF
    l[3, 10] = l[3, 60] = INF               # two of +inf share the softmax
    l[5] = torch.finfo(torch.float32).min   # a mask of the type's lowest value is still a logit
    l[6, 1:] = torch.finfo(torch.float32).min
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            assert check(l, 8, scoring=scoring, renormalize=renormalize) == 0
    l[4, ::2] = NAN
    l[7] = NAN
    for renormalize in (True, False):
        assert check(l, 8, renormalize=renormalize) == ep.EP_FLAG_BAD_LOGIT
    assert check(l, 8, scoring="sigmoid", groups=7, groups_per_token=2) == ep.EP_FLAG_BAD_LOGIT


def test_route_bias_chooses_only():
    l = logits_of(50, 128, torch.float32, 9)
    bias = torch.zeros(128, device=DEV)
    bias[5], bias[9], bias[17] = 100.0, -INF, INF
    assert check(l, 8, bias=bias) == 0
    idx, w = ep.route(l, 8, bias=bias)
    assert (idx[:, 0] == 17).all() and (idx[:, 1] == 5).all() and not (idx == 9).any()
    # weights come from the logits alone, far below the row's maximum here
    l[:, 5] = l[:, 17] = -200.0
    l[:, 30] = 200.0
    assert check(l, 2, bias=bias) == 0
    bias[3] = NAN
    assert check(l, 2, bias=bias) == ep.EP_FLAG_BAD_LOGIT


def test_route_sigmoid_of_very_negative_logits():
    l = torch.full((3, 16), -1.0e4, device=DEV)
    l[1, 4] = -80.0
    assert check(l, 4, scoring="sigmoid") == 0


def test_route_writes_only_its_outputs_on_the_given_stream():
    l = logits_of(37, 96, torch.bfloat16)
    raw_i = torch.full((37 * 6 + 64,), -7, dtype=torch.int32, device=DEV)
    raw_w = torch.full((37 * 6 + 64,), -7.0, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        idx, w = ep.route(l, 6, topk_idx=raw_i[32:32 + 37 * 6].view(37, 6), topk_w=raw_w[32:32 + 37 * 6].view(37, 6))
    s.synchronize()
    assert torch.equal(idx.cpu().long(), ref.route(l, 6)[0])
    for raw in (raw_i, raw_w):
        assert (raw[:32] == -7).all() and (raw[-32:] == -7).all()


def test_route_feeds_the_layout_and_replays_in_a_graph():
    l = logits_of(300, 128, torch.float32, 1)
    idx, w = torch.zeros(300, 8, dtype=torch.int32, device=DEV), torch.zeros(300, 8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        ep.route(l, 8, topk_idx=idx, topk_w=w)
        lay = ep.layout(idx, 128)
    l.copy_(logits_of(300, 128, torch.float32, 2))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx.cpu().long(), ref.route(l, 8)[0])
    assert torch.equal(lay.expert_counts.cpu().long(), torch.bincount(idx.cpu().long().view(-1), minlength=128))


def test_route_beyond_32_bit_offsets():
    T, E = (1 << 23) + 5, 512                     # 2^32 logits and some
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(T, device=DEV) % E
    l.scatter_(1, at[:, None], 3.0)
    idx, w = ep.route(l, 1)
    assert torch.equal(idx[:, 0].long(), at) and (w == 1.0).all()


def test_route_of_no_tokens():
    idx, w = ep.route(torch.empty(0, 64, device=DEV), 8)
    assert idx.shape == (0, 8) and w.shape == (0, 8)


def test_route_refusals():
    l = logits_of(4, 64, torch.float32)
    for bad in (dict(scoring="other"), dict(bias=torch.zeros(63, device=DEV)), dict(bias=torch.zeros(64)),
                dict(topk_idx=torch.zeros(4, 7, dtype=torch.int32, device=DEV)),
                dict(topk_w=torch.zeros(4, 8, dtype=torch.float16, device=DEV))):
        with pytest.raises(ValueError):
            ep.route(l, 8, **bad)
    with pytest.raises(ValueError):
        ep.route(l.half(), 8)
    with pytest.raises(ValueError):
        ep.route(l.t(), 2)
    for bad in (dict(k=65), dict(k=8, groups=3), dict(k=8, groups=64), dict(k=8, groups=4, groups_per_token=5),
                dict(k=8, groups=4, groups_per_token=0)):
        with pytest.raises(ep.EpError):
            ep.route(l, **bad)
