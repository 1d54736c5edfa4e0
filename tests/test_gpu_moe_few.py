"""The whole expert layer for a few tokens (ep_moe_few) against a plain 64-bit
definition, and against the chain of dispatch, both products and combine."""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import moe_reference as ref
from gpu_helpers import DEV
from test_gpu_group_gemm import gen, random_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def problem(T, H, I, E, k, seed, idx=None):
    g = gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    sc = lambda *s: 0.75 + 0.5 * torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    if idx is None:
        idx = torch.topk(rnd(T, E), k, dim=1).indices.to(torch.int32)
    return dict(x=rnd(T, H).to(torch.bfloat16), topk_idx=idx, topk_w=torch.softmax(rnd(T, k), dim=1),
                w13_q=random_codes((E, 2 * I, H), g), w13_scale=sc(E, 2 * I // 128, H // 128) / 100 * H ** -0.5,
                w2_q=random_codes((E, H, I), g), w2_scale=sc(E, H // 128, I // 128) / 100 * I ** -0.5)


def expected(p, reciprocal=True):
    """(out in 64 bits, bound), x cast as ep_moe_few or as ep_dispatch_fp8 does: the fp32 errors of both products, of SwiGLU and
    of the sum over experts, and what the cast of h can be off where they move
    a value across a midpoint of e4m3 (carried through |w2|)."""
    T, H = p["x"].shape
    I = p["w2_q"].shape[2]
    E = p["w2_q"].shape[0]
    xq, xs = ref.quantise_f32(p["x"], reciprocal)
    x = xq * xs.double().repeat_interleave(128, dim=1)
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(E):
        t, j = torch.nonzero(p["topk_idx"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w13 = ref.weights64(p["w13_q"][e], p["w13_scale"][e])
        y, dy = x[t] @ w13.T, ref.gamma(H) * (x[t].abs() @ w13.abs().T)
        h, dh = ref.silu_mul(y[:, :I], y[:, I:], dy[:, :I], dy[:, I:])
        hq, slack, _, _ = ref.flip_slack(h, dh)
        w2 = ref.weights64(p["w2_q"][e], p["w2_scale"][e])
        wt = p["topk_w"][t, j].double()[:, None]
        part = wt * (hq @ w2.T)
        out.index_add_(0, t, part)
        err.index_add_(0, t, wt.abs() * (slack @ w2.abs().T + ref.gamma(I) * (hq.abs() @ w2.abs().T)))
        mag.index_add_(0, t, part.abs())
    k = p["topk_idx"].shape[1]
    return out, err + ref.gamma(16 + k) * mag  # sixteen partial sums and k experts


def check(p, status=0):
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    T, H = p["x"].shape
    raw = torch.full((T * H + 128,), -7.0, dtype=torch.bfloat16, device=DEV)
    got = ep.moe_few(**p, out=raw[64:-64].view(T, H), status=word)
    assert ep.status_read(word) == status
    again = ep.moe_few(**p)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))  # the same bits every time
    assert (raw[:64] == -7).all() and (raw[-64:] == -7).all()
    want, err = expected(p)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (want.abs() + err) + err).all()
    return got, want


@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 1, 1), (1, 2048, 1024, 128, 8), (2, 7168, 2048, 16, 8),
                                       (3, 384, 640, 60, 6), (8, 1024, 256, 8, 2), (9, 128, 384, 4, 4),
                                       (17, 896, 128, 64, 8), (33, 2048, 768, 128, 8), (45, 640, 1408, 16, 4),
                                       (64, 512, 256, 3, 3), (64, 1152, 384, 256, 8), (64, 256, 128, 1024, 32),
                                       (5, 16384, 128, 4, 2), (5, 128, 16384, 4, 2)])
def test_matches_the_definition(T, H, I, E, k):
    check(problem(T, H, I, E, k, T + H))


def test_dropped_pairs_empty_tokens_and_bad_ids():
    p = problem(12, 512, 256, 16, 4, 1)
    p["topk_idx"][0] = -1                     # nothing: +0
    p["topk_idx"][1, 1:] = -1
    p["topk_idx"][5, 2] = -1
    got, _ = check(p)
    assert (got[0].view(torch.int16) == 0).all()
    p["topk_idx"][3, 0], p["topk_idx"][4, 1] = 16, -5
    q = dict(p)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = ep.moe_few(**p, status=word)
    assert ep.status_read(word) == ep.EP_FLAG_BAD_EXPERT
    q["topk_idx"] = torch.where((p["topk_idx"] < 0) | (p["topk_idx"] >= 16), -1, p["topk_idx"])
    assert torch.equal(got, ep.moe_few(**q))
    q["topk_idx"] = torch.full_like(p["topk_idx"], -1)   # no pair at all
    assert (ep.moe_few(**q).view(torch.int16) == 0).all()


def test_every_token_to_one_expert_and_a_token_with_an_expert_twice():
    idx = torch.zeros(64, 2, dtype=torch.int32, device=DEV)
    idx[:, 1] = 3
    check(problem(64, 256, 256, 4, 2, 2, idx))
    idx = torch.full((40, 6), 2, dtype=torch.int32, device=DEV)   # 240 pairs of one expert
    check(problem(40, 128, 128, 4, 6, 3, idx))


def test_zero_and_extreme_rows():
    p = problem(6, 512, 256, 8, 4, 4)
    p["x"][1] = 0
    p["x"][2] *= 1.0e4
    p["x"][3, 100:300] = 0
    p["topk_w"][4] = 0.0
    check(p)


def test_agrees_with_the_chain():
    T, H, I, E, k = 50, 1024, 512, 32, 8
    p = problem(T, H, I, E, k, 5)
    lay, q, s = ep.layout_dispatch(p["x"], p["topk_idx"], E, fp8=True)
    hq, hs = ep.group_gemm_swiglu_fp8(q, s, p["w13_q"], p["w13_scale"], lay.expert_counts, lay.expert_offsets)
    y = ep.group_gemm_fp8(hq, hs, p["w2_q"], p["w2_scale"], lay.expert_counts, lay.expert_offsets)
    chain = ep.combine(y, p["topk_w"], lay.dst_row)
    got = ep.moe_few(**p)
    # Both hold `expected`'s bound for their cast of x; the chain also rounds
    # each y to bf16 (2^-8 of it) before the weighted sum.
    want, err = expected(p, reciprocal=False)
    ysum = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for j in range(k):
        ysum += p["topk_w"][:, j:j + 1].double().abs() * y[lay.dst_row[:, j].long()].double().abs()
    assert ((chain.double() - want).abs() <= 2.0 ** -8 * (want.abs() + ysum * 1.01 + err) + err).all()
    want, err = expected(p)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (want.abs() + err) + err).all()


def test_graph_replay_with_new_inputs_on_another_stream():
    p = problem(7, 512, 256, 16, 4, 6)
    out = torch.zeros_like(p["x"])
    ws = torch.zeros(ep.moe_few_workspace_bytes(7, 4, 256), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        ep.moe_few(**p, out=out, workspace=ws)
    p["x"].copy_(problem(7, 512, 256, 16, 4, 7)["x"])
    p["topk_idx"].copy_(problem(7, 512, 256, 16, 4, 8)["topk_idx"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ep.moe_few(**p))


def test_no_tokens_and_refusals():
    p = problem(4, 256, 128, 4, 2, 9)
    e = {**p, "x": p["x"][:0], "topk_idx": p["topk_idx"][:0], "topk_w": p["topk_w"][:0]}
    assert ep.moe_few(**e).shape == (0, 256)
    for name, bad in (("x", p["x"].float()), ("topk_idx", p["topk_idx"].long()), ("topk_w", p["topk_w"][:, :1].contiguous()),
                      ("w13_q", p["w13_q"][:, :128].contiguous()), ("w2_scale", p["w2_scale"][:, :1].contiguous()),
                      ("w2_q", p["w2_q"].transpose(1, 2)), ("out", torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            ep.moe_few(**{**p, name: bad})
    with pytest.raises(ep.EpError):
        ep.moe_few(**p, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ep.EpError):
        ep.moe_few(**problem(65, 256, 128, 4, 2, 10))
