"""The expert layer takes the same weights for every number of tokens, also
where its few-token call does not."""
import os
import re

import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV
from test_gpu_expert_layer import layer_of
from test_gpu_moe_few import expected, problem


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_width_limit_matches_the_header():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep.h")) as f:
        assert int(re.search(r"#define EP_MOE_FEW_MAX_WIDTH (\d+)", f.read()).group(1)) == ep.MOE_FEW_MAX_WIDTH


def check_long(layer, p):
    """One expert per token: the longer path's result is bf16 of bf16's y times its weight."""
    out = layer.experts(p["x"], p["topk_idx"], p["topk_w"])
    assert ep.status_read(layer.status) == 0
    assert out.shape == p["x"].shape
    if out.numel() == 0:
        return
    want, err = expected(p, reciprocal=False)
    # y is rounded to bf16 (2^-8 of it) before the weight, the sum once more
    assert ((out.double() - want).abs() <= 2.0 ** -8 * (want.abs() * 2.01 + 2 * err) + err).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 65])
@pytest.mark.parametrize("H,I", [(128, 16512), (16512, 128)])
def test_widths_beyond_the_few_token_call(built, T, H, I):
    p = problem(T, H, I, 2, 1, 7)
    layer = layer_of(p, 1)
    assert not layer.few(T)
    check_long(layer, p)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 65])
@pytest.mark.parametrize("name", ["w13_q", "w2_q"])
def test_weights_on_16_but_not_32_bytes(built, T, name):
    p = problem(T, 256, 128, 4, 1, 9)
    raw = torch.empty(p[name].numel() + 32, dtype=torch.uint8, device=DEV)
    moved = raw[16:16 + p[name].numel()].view(p[name].shape)
    moved.copy_(p[name])
    assert moved.data_ptr() % 32 == 16
    p[name] = moved
    layer = layer_of(p, 1)
    assert not layer.few(T)
    check_long(layer, p)


@pytest.mark.gpu
def test_widest_layer_of_the_few_token_call(built):
    p = problem(1, 128, ep.MOE_FEW_MAX_WIDTH, 2, 1, 11)
    assert layer_of(p, 1).few(1)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 100])     # one for each path
def test_shapes_are_refused_on_both_paths(built, T):
    p = problem(T, 256, 128, 8, 2, 13)
    layer = layer_of(p, 2)
    assert layer.few(T) == (T == 4)
    x, idx, w = p["x"], p["topk_idx"], p["topk_w"]
    for args in ((x, idx[:, :1].contiguous(), w), (x, idx, w[:, :1].contiguous()), (x, idx[1:], w[1:]),
                 (x[1:], idx, w), (x, idx, w[1:]), (x[:, :128].contiguous(), idx, w), (x, idx.view(-1), w.view(-1)),
                 (x, idx, w, torch.empty(T - 1, 256, dtype=torch.bfloat16, device=DEV)),
                 (x, idx, w, torch.empty(T, 128, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            layer.experts(*args)


@pytest.mark.gpu
def test_weights_that_do_not_fit_each_other_are_refused(built):
    p = problem(1, 256, 128, 4, 2, 17)
    for w2 in (p["w2_q"][:3], p["w2_q"][:, :128].contiguous(), p["w2_q"][:, :, :64].contiguous()):
        with pytest.raises(ValueError):
            ep.ExpertLayer(p["w13_q"], p["w13_scale"], w2, p["w2_scale"], 2)
