"""The expert layer from logits to combined hidden states: both of its paths
against the plain 64-bit definition, and against the calls that it makes."""
import os
import subprocess
import sys

import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import moe_reference as ref
from gpu_helpers import DEV
from test_gpu_group_gemm import gen
from test_gpu_moe_few import expected, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def layer_of(p, k, **kw):
    return ep.ExpertLayer(p["w13_q"], p["w13_scale"], p["w2_q"], p["w2_scale"], k, **kw)


@pytest.mark.parametrize("T", [1, 37, 64, 65, 200])
def test_both_paths_match_the_definition(T):
    H, I, E, k = 512, 384, 16, 4
    p = problem(T, H, I, E, k, T)
    logits = torch.randn(T, E, generator=gen(T), device=DEV)
    layer = layer_of(p, k, groups=4, groups_per_token=2)
    out = layer(p["x"], logits)
    idx, w = ref.route(logits, k, groups=4, groups_per_token=2)
    few = layer.few(T)  # the two paths cast x with another quotient
    want, err = expected({**p, "topk_idx": idx.to(DEV), "topk_w": w.to(DEV)}, few)
    # the longer path rounds each expert's output to bf16 (2^-8 of it), at most
    # the sum of the magnitudes of its terms; the weights are good to 2^-16
    terms = torch.zeros_like(want)
    for j in range(k):
        one = {**p, "topk_idx": idx[:, j:j + 1].to(DEV), "topk_w": w[:, j:j + 1].to(DEV)}
        terms += expected(one, few)[0].abs()
    bound = 2.0 ** -8 * (want.abs() + 1.01 * terms + err) + err + 2.0 ** -16 * terms
    assert ((out.double() - want).abs() <= bound).all()
    assert ep.status_read(layer.status) == 0


def test_choice_of_the_path():
    p = problem(1, 256, 128, 8, 2, 3)
    small = layer_of(p, 2)
    assert small.few(1) and small.few(64) and not small.few(65)
    big = layer_of({**p, "w13_q": p["w13_q"].expand(8, 256, 256)}, 2)
    big.w13_q = torch.empty(8, 4096, 2048, dtype=torch.uint8, device=DEV)  # 64 MB of weights
    assert big.few(8) and not big.few(9)


def test_flags_of_every_call_reach_the_status_word():
    p = problem(100, 256, 128, 8, 2, 1)
    layer = layer_of(p, 2)
    idx = p["topk_idx"].clone()
    idx[3, 1] = 77
    layer.experts(p["x"], idx, p["topk_w"])
    assert ep.status_read(layer.status) == ep.EP_FLAG_BAD_EXPERT
    layer.status.zero_()
    layer.experts(p["x"][:8], idx[:8].contiguous(), p["topk_w"][:8].contiguous())
    assert ep.status_read(layer.status) == ep.EP_FLAG_BAD_EXPERT


def test_refusals():
    p = problem(4, 256, 128, 8, 2, 2)
    with pytest.raises(ValueError):
        ep.ExpertLayer(p["w13_q"], p["w13_scale"], p["w2_q"][:, :, :64], p["w2_scale"], 2)
    with pytest.raises(ValueError):
        layer_of(p, 2)(p["x"], torch.zeros(4, 9, device=DEV))


def test_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "expert_layer.py"), "--hidden", "512",
                        "--inner", "256", "--experts", "16", "--topk", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-2000:]
    assert r.stdout.count("us per layer") == 3


CAPTURE = r'''
import sys, torch
sys.path.insert(0, ROOT_DIR)
import combine_ep_layout_02_gb300 as ep
dev = torch.device("cuda:0")
E, H, I, k = 8, 256, 128, 2
g = torch.Generator(device=dev).manual_seed(1)
codes = lambda *s: torch.randint(0, 127, s, generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
layer = ep.ExpertLayer(codes(E, 2 * I, H), torch.full((E, 2, 2), 1e-4, device=dev), codes(E, H, I),
                       torch.full((E, 2, 1), 1e-4, device=dev), k)
for T in (5, 100):
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device=dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        out = layer(x, logits)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer(x, logits)) and ep.status_read(layer.status) == 0
print("CAPTURE-FIRST OK")
'''


def test_first_calls_inside_graph_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE.replace("ROOT_DIR", repr(root))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "CAPTURE-FIRST OK" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
