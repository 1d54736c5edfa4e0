"""Host-side argument checks of the router and the expert products (no GPU
needed: every call below is refused before anything is enqueued)."""
import ctypes
import os
import re

import pytest

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced


def off(n):
    return ctypes.c_void_p((1 << 20) + n)


@pytest.fixture(scope="module")
def lib():
    from combine_ep_layout_02_gb300 import build as cuda_build
    cuda_build.build()
    from combine_ep_layout_02_gb300 import binding
    return binding.load()


def test_limits_match_the_header():
    from combine_ep_layout_02_gb300 import binding
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep.h")) as f:
        text = f.read()
    assert int(re.search(r"#define EP_MOE_FEW_MAX_TOKENS (\d+)", text).group(1)) == binding.MOE_FEW_MAX_TOKENS
    assert int(re.search(r"EP_TYPE_BF16 = (\d)", text).group(1)) == 1
    assert int(re.search(r"EP_SCORE_SIGMOID = (\d)", text).group(1)) == binding.SCORES["sigmoid"]


def test_route_argument_validation(lib):
    def call(logits=FAKE, ty=0, bias=None, T=4, E=64, k=8, groups=1, gpt=1, score=0, idx=FAKE, w=FAKE, status=None):
        return lib.ep_route(logits, ty, bias, T, E, k, groups, gpt, score, 1, 1.0, idx, w, status, None)
    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(E=0) == 1 and call(E=1025) == 1
    assert call(k=0) == 1 and call(k=33) == 1 and call(E=4, k=5) == 1
    assert call(T=1 << 30, k=8) == 1
    assert call(groups=0) == 1 and call(groups=33, E=66) == 1 and call(groups=5) == 1
    assert call(groups=4, gpt=0) == 1 and call(groups=4, gpt=5) == 1
    assert call(ty=2) == 1 and call(score=2) == 1 and call(ty=-1) == 1
    assert call(logits=None) == 1 and call(idx=None) == 1 and call(w=None) == 1
    assert call(logits=off(2)) == 2 and call(ty=1, logits=off(1)) == 2
    assert call(bias=off(2)) == 2 and call(idx=off(2)) == 2 and call(w=off(1)) == 2 and call(status=off(2)) == 2


@pytest.mark.parametrize("swiglu", [False, True])
def test_group_gemm_argument_validation(lib, swiglu):
    def call(a=FAKE, s=FAKE, rows=64, K=256, w=FAKE, ws=FAKE, N=128, E=4, cnt=FAKE, offs=FAKE, kind=0, cap=0,
             out=FAKE, scale=FAKE, status=None):
        if swiglu:
            return lib.ep_group_gemm_swiglu_fp8(a, s, rows, K, w, ws, N, E, cnt, offs, kind, cap, out, scale, status,
                                                None)
        return lib.ep_group_gemm_fp8(a, s, rows, K, w, ws, N, E, cnt, offs, kind, cap, out, status, None)
    assert call(rows=0, a=None, s=None) == 0
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(K=0) == 1 and call(N=0) == 1 and call(E=0) == 1 and call(E=1025) == 1
    assert call(E=1024, N=1 << 21) == 1             # weight rows beyond 31 bits
    assert call(K=200) == 2
    assert call(N=100 if not swiglu else 64) == 2
    assert call(kind=2) == 1 and call(kind=1, cap=-1) == 1 and call(kind=1, cap=17) == 1
    assert call(a=None) == 1 and call(s=None) == 1 and call(w=None) == 1 and call(ws=None) == 1
    assert call(cnt=None) == 1 and call(offs=None) == 1 and call(out=None) == 1
    assert call(a=off(8)) == 2 and call(w=off(8)) == 2 and call(out=off(8)) == 2
    assert call(s=off(2)) == 2 and call(ws=off(2)) == 2 and call(cnt=off(1)) == 2 and call(offs=off(2)) == 2
    assert call(status=off(2)) == 2
    if swiglu:
        assert call(scale=None) == 1 and call(scale=off(2)) == 2


def test_moe_few_argument_validation(lib):
    def call(x=FAKE, T=4, H=256, k=2, idx=FAKE, w=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, I=128, E=8, out=FAKE,
             status=None, ws=FAKE, wsb=1 << 20):
        return lib.ep_moe_few(x, T, H, k, idx, w, w13, s13, w2, s2, I, E, out, status, ws, wsb, None)
    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(T=65) == 1
    assert call(H=0) == 1 and call(H=16512) == 1 and call(I=0) == 1 and call(I=16512) == 1
    assert call(k=0) == 1 and call(k=33) == 1 and call(E=0) == 1 and call(E=1025) == 1
    assert call(H=200) == 2 and call(I=64) == 2
    for name in ("x", "idx", "w", "w13", "s13", "w2", "s2", "out"):
        assert call(**{name: None}) == 1, name
    for name, n in (("x", 8), ("idx", 2), ("w", 2), ("w13", 16), ("s13", 2), ("w2", 16), ("s2", 2), ("out", 8),
                    ("status", 2), ("ws", 8)):
        assert call(**{name: off(n)}) == 2, name
    need = lib.ep_moe_few_workspace_bytes(4, 2, 128)
    assert need >= 4 * 2 * 128 + 4 * 2 * 4 and lib.ep_moe_few_workspace_bytes(0, 2, 128) == 0
    assert call(ws=None) == 3 and call(wsb=need - 1) == 3
