"""Host-side argument checks of the BF16 products, the dense layer and the
combine's gradient (no GPU needed: every call below is refused before anything
is enqueued)."""
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


def test_names_match_the_header():
    from combine_ep_layout_02_gb300 import binding
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep.h")) as f:
        text = f.read()
    found = {n.lower(): int(v) for n, v in re.findall(r"\bEP_ACT_(\w+) = (\d)", text)}
    assert found == binding.ACTIVATIONS
    assert [binding.TYPES[t] for t in binding.TYPES] == [0, 1]
    assert int(re.search(r"#define EP_LINEAR_FEW_TOKENS (\d+)", text).group(1)) == binding.LINEAR_FEW_TOKENS


GROUP = ["forward", "swiglu", "dgrad", "swiglu_dgrad", "wgrad"]


@pytest.mark.parametrize("which", GROUP)
def test_group_argument_validation(lib, which):
    def call(a=FAKE, rows=64, K=256, w=FAKE, N=128, E=4, cnt=FAKE, offs=FAKE, kind=0, cap=0, out=FAKE, z=FAKE,
             ty=1, status=None):
        seg = (cnt, offs, kind, cap)
        if which == "forward":
            return lib.ep_group_gemm(a, rows, K, w, N, E, *seg, out, status, None)
        if which == "swiglu":
            return lib.ep_group_gemm_swiglu(a, rows, K, w, N, E, *seg, out, z, status, None)
        if which == "dgrad":
            return lib.ep_group_gemm_dgrad(a, rows, K, w, N, E, *seg, out, status, None)
        if which == "swiglu_dgrad":
            return lib.ep_group_gemm_swiglu_dgrad(a, rows, K, w, N, E, z, *seg, out, status, None)
        return lib.ep_group_gemm_wgrad(a, w, rows, N, K, E, *seg, z, out, ty, status, None)
    if which != "wgrad":
        assert call(rows=0, a=None) == 0
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1 and call(rows=(1 << 31) - 256) == 1
    assert call(N=(1 << 30) + 16, E=1) == 1 and call(K=(1 << 30) + 16, E=1) == 1
    assert call(K=0) == 1 and call(N=0) == 1 and call(E=0) == 1 and call(E=1025) == 1
    assert call(E=1024, N=1 << 21, K=1 << 21) == 1      # weight rows beyond 31 bits
    assert call(K=100) == 2 and call(N=100) == 2
    if "swiglu" in which:
        assert call(N=24) == 2
    assert call(kind=2) == 1 and call(kind=-1) == 1 and call(kind=1, cap=-1) == 1 and call(kind=1, cap=17) == 1
    for name in ("a", "w", "cnt", "offs", "out"):
        assert call(**{name: None}) == 1, name
    if which == "swiglu_dgrad":
        assert call(z=None) == 1
    for name, n in (("a", 8), ("w", 8), ("out", 8), ("cnt", 1), ("offs", 2), ("status", 2)):
        assert call(**{name: off(n)}) == 2, name
    if which in ("swiglu", "swiglu_dgrad", "wgrad"):
        assert call(z=off(8)) == 2
    if which == "wgrad":
        assert call(ty=2) == 1 and call(ty=-1) == 1


def test_linear_argument_validation(lib):
    def call(x=FAKE, M=4, K=64, w=FAKE, N=64, bias=None, bt=0, act=0, res=None, out=FAKE, ty=1, z=None, status=None,
             ws=FAKE, wsb=1 << 30):
        return lib.ep_linear(x, M, K, w, N, bias, bt, act, res, out, ty, z, status, ws, wsb, None)
    assert call(M=0, x=None, out=None) == 0
    assert call(M=-1) == 1 and call(M=(1 << 31) - 256) == 1 and call(K=0) == 1 and call(N=0) == 1
    assert call(N=(1 << 30) + 8) == 1 and call(K=(1 << 30) + 8) == 1 and call(N=(1 << 29) + 16, act=4) == 1
    assert call(act=5) == 1 and call(act=-1) == 1 and call(ty=2) == 1 and call(bt=2) == 1 and call(act=4, ty=0) == 1
    assert call(K=60) == 2 and call(N=60) == 2 and call(act=4, N=24) == 2
    for name in ("x", "w", "out"):
        assert call(**{name: None}) == 1, name
    for name, n in (("x", 8), ("w", 8), ("out", 8), ("res", 8), ("z", 8), ("bias", 2), ("status", 2)):
        assert call(**{name: off(n)}) == 2, name
    assert call(bias=off(1), bt=1) == 2
    assert lib.ep_linear_workspace_bytes(0, 64, 64, 0) == 0


def test_linear_backward_argument_validation(lib):
    def call(dy=FAKE, x=FAKE, w=FAKE, z=FAKE, M=4, K=64, N=64, act=2, dz=FAKE, dx=FAKE, add=None, dw=FAKE, ty=0,
             db=FAKE, status=None, ws=FAKE, wsb=1 << 40):
        return lib.ep_linear_backward(dy, x, w, z, M, K, N, act, dz, dx, add, dw, ty, db, status, ws, wsb, None)
    assert lib.ep_linear_backward_workspace_bytes(4, 64, 64, 2) == 0
    assert call(M=-1) == 1 and call(M=1 << 31) == 1 and call(K=0) == 1 and call(N=0) == 1
    assert call(act=5) == 1 and call(ty=2) == 1
    assert call(K=60) == 2 and call(N=60) == 2 and call(act=4, N=24) == 2
    assert call(z=None) == 1 and call(dz=None) == 1 and call(act=0) == 1 and call(act=0, z=None) == 1
    assert call(dy=None) == 1 and call(x=None) == 1 and call(w=None) == 1
    for name, n in (("dy", 8), ("x", 8), ("w", 8), ("z", 8), ("dz", 8), ("dx", 8), ("add", 8), ("dw", 8), ("db", 2),
                    ("status", 2)):
        assert call(**{name: off(n)}) == 2, name


def test_combine_backward_argument_validation(lib):
    def call(dout=FAKE, y=FAKE, w=FAKE, dst=FAKE, T=4, H=64, k=2, rows=8, dy=FAKE, dw=FAKE, status=None):
        return lib.ep_combine_backward(dout, y, w, dst, T, H, k, rows, dy, dw, status, None)
    assert call(T=0, dout=None) == 0
    assert call(T=-1) == 1 and call(H=0) == 1 and call(k=0) == 1 and call(k=33) == 1 and call(rows=-1) == 1
    assert call(T=1 << 30) == 1 and call(H=60) == 2
    for name in ("dout", "w", "dst", "dy", "y"):
        assert call(**{name: None}) == 1, name
    for name, n in (("dout", 8), ("y", 8), ("dy", 8), ("w", 2), ("dw", 2), ("dst", 2), ("status", 2)):
        assert call(**{name: off(n)}) == 2, name
