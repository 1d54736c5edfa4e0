"""Long sums of the BF16 products and the dense layer.  The operands are positive,
so that a sum that is truncated at every step shrinks instead of hiding among
errors of both signs, and spread over eight binades, so that no step is exact.

Bounds, in parts of 2^-24 of the result.  An addition that truncates loses less than
an ulp of the sum, at most 2 parts of it, and half of that on average.  Over n
additions of positive products the sum grows in proportion: sum over i of 2 i / n =
n + 1 parts at most, (n + 1) / 2 on average.
  * A sum that ends after 512 values has 512 additions: a step of the tensor core
    adds 16 products to the sum, and each of these may be cut to the sum's ulp.
  * P such sums added with rounding: half an ulp, one part, of each of the growing
    sums, (P + 1) / 2 together, and of both signs, so that a mean over the outputs
    keeps less than one part of it.  One part more for a last rounding (bias, finish).
  * A bf16 output of at most 16,384 values may come from one sum.
(A sum of n values that is cut nowhere was seen to lose n / 16 to n / 20 parts.)
"""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

import product_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
PART = 512


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def positive(*shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    v = 1 + torch.rand(*shape, generator=g, device=DEV)
    return (v * torch.exp2(-torch.randint(0, 8, shape, generator=g, device=DEV).float())).to(BF16)


def product(a, b):
    """a [m, k], b [n, k] in 64 bits, by pieces."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=DEV)
    for k in range(0, a.shape[1], 1 << 16):
        out += a[:, k:k + (1 << 16)].double() @ b[:, k:k + (1 << 16)].double().T
    return out


def parts(n):
    # warps and blocks share a sum in up to 64 slices, each of whose last part may be short
    return -(-n // 512) + 64


def check_f32(got, want, n):
    assert got.dtype is F32
    off = (got.double() - want) / want / U
    assert off.mean().abs() <= (PART + 1) / 2 + 2, float(off.mean())
    assert off.abs().max() <= PART + 1 + (parts(n) + 1) / 2 + 1, float(off.abs().max())


def check_bf16(got, want, n, whole=0):
    assert got.dtype is BF16
    lost = n if n <= whole else PART + (parts(n) + 1) / 2
    assert ref.close(got, want, (lost + 2) * U * want), float(((got.double() - want) / want / U).abs().max())


def one(n):
    return torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("K", [512, 4096, 7168, 16384, 65536])
@pytest.mark.parametrize("M,N", [(1, 256), (1, 6000), (8, 256), (8, 6000), (12, 256), (16, 6000), (24, 256), (24, 6000),
                                 (32, 6000), (40, 256), (300, 256), (300, 6000)])
def test_dense_float32_outputs(M, N, K):
    x, w = positive(M, K), positive(N, K, seed=1)
    check_f32(ep.linear(x, w, dtype=F32), product(x, w), K)


@pytest.mark.parametrize("rows", [512, 1000, 4096, 16384, 65536, 1 << 18])
def test_weight_gradients_in_float32(rows):
    dy, x = positive(rows, 264), positive(rows, 136, seed=1)
    want = product(dy.T.contiguous(), x.T.contiguous())
    check_f32(ep.group_gemm_wgrad(dy, x, *one(rows))[0], want, rows)
    check_f32(ep.linear_backward(dy, x, positive(264, 136), with_dx=False).dw, want, rows)


@pytest.mark.parametrize("rows", [1000, 1 << 16, 1 << 20, 1 << 22])
def test_weight_gradients_in_bf16(rows):
    dy, x = positive(rows, 136), positive(rows, 72, seed=1)
    want = product(dy.T.contiguous(), x.T.contiguous())
    check_bf16(ep.group_gemm_wgrad(dy, x, *one(rows), dtype=BF16)[0], want, rows)
    check_bf16(ep.linear_backward(dy, x, positive(136, 72), dtype=BF16, with_dx=False, with_dbias=False).dw, want, rows)


@pytest.mark.parametrize("n", [7168, 16384, 16392, 1 << 18, 1 << 20])
@pytest.mark.parametrize("M", [7, 300])
def test_products_of_a_long_summed_index(M, n):
    whole = 16384
    x, w = positive(M, n), positive(1, 160, n, seed=1)
    want = product(x, w[0])
    check_bf16(ep.group_gemm(x, w, *one(M))[:M], want, n, whole)
    z = torch.empty(M, 160, dtype=BF16, device=DEV)
    h = ep.group_gemm_swiglu(x, w, *one(M), z=z)
    check_bf16(z, want, n, whole)
    lost = (n if n <= whole else PART + (parts(n) + 1) / 2) + 2
    y, off = ref.gated(want, lost * U * want)
    assert ref.close(h, y, off)
    wt = w.transpose(1, 2).contiguous()
    check_bf16(ep.group_gemm_dgrad(x, wt, *one(M)), want, n, whole)
    z2 = positive(M, 320, seed=2)
    dz = ep.group_gemm_swiglu_dgrad(x, wt, z2, *one(M))
    assert ref.close(dz, *ref.gated_back(z2.double(), want, lost * U * want))


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("M,N", [(40, 4096), (300, 4096), (3000, 4096)])
def test_dense_layers_of_a_long_summed_index(M, N, act):
    """Epilogues of long sums: cut between blocks (two parts and a second pass) or within a tile."""
    K = 16384 + 64
    g = torch.Generator(device=DEV)
    g.manual_seed(5)

    def normal(*shape, amp=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * amp).to(BF16)

    rows = 2 * N if act == "swiglu" else N
    x, w, bias, res = normal(M, K), normal(rows, K, amp=K ** -0.5), normal(rows), normal(M, N)
    z = torch.empty(M, rows, dtype=BF16, device=DEV)
    out = ep.linear(x, w, bias=bias, activation=act, residual=res, z=z)
    want, off, y, dy = ref.linear(x, w, bias, act, res)
    assert ref.close(out, want, off) and ref.close(z, y, dy)


@pytest.mark.parametrize("M,rows", [(1, 512), (8, 512), (16, 512), (24, 512), (24, 5120)])
def test_few_tokens_with_a_very_long_summed_index(M, rows):
    K = 8 * 16384 + 1032  # beyond the longest sum that is never cut
    x, w = positive(M, K), positive(rows, K, seed=1)
    want = product(x, w)
    z = torch.empty(M, rows, dtype=BF16, device=DEV)
    check_bf16(ep.linear(x, w, z=z), want, K)
    check_bf16(z, want, K)
    check_f32(ep.linear(x, w, dtype=F32), want, K)
    y, off = ref.gated(want, (PART + (parts(K) + 1) / 2 + 2) * U * want)
    assert ref.close(ep.linear(x, w, activation="swiglu"), y, off)
