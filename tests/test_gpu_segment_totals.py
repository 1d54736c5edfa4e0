"""Segments that overlap so much that their tiles pass 31 bits are reported, and
nothing is computed for them.  (The buffers are not touched: no row of theirs is
read or written.)"""
import pytest
import torch

import combine_ep_layout_02_gb300 as ep

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

E = 1024


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def needs(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("needs %d GB" % gigabytes)


def segments(rows):
    return (torch.full((E,), rows, dtype=torch.int32, device=DEV), torch.zeros(E, dtype=torch.int32, device=DEV))


def test_bf16_products():
    needs(40)
    rows = (1 << 29) + 4096     # 2^21 + 16 tiles of 256 rows, 1,024 times
    x = torch.empty(rows, 8, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(rows, 8, dtype=torch.bfloat16, device=DEV)
    x[:16], out[:16], out[-16:] = 1, 5, 5
    w = torch.ones(E, 8, 8, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in (lambda: ep.group_gemm(x, w, *segments(rows), out=out, status=status),
                 lambda: ep.group_gemm_dgrad(x, w, *segments(rows), dx=out, status=status)):
        status.zero_()
        call()
        assert ep.status_read(status) == ep.EP_FLAG_BAD_ROW
        assert (out[:16] == 5).all() and (out[-16:] == 5).all()


def test_fp8_products():
    needs(60)
    rows = (1 << 28) + 4096     # 2^21 + 32 tiles of 128 rows
    a = torch.empty(rows, 128, dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, 1, device=DEV)
    w, ws = torch.zeros(E, 8, 128, dtype=torch.uint8, device=DEV), torch.ones(E, 1, 1, device=DEV)
    out = torch.empty(rows, 8, dtype=torch.bfloat16, device=DEV)
    out[:16], out[-16:] = 5, 5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ep.group_gemm_fp8(a, s, w, ws, *segments(rows), out=out, status=status)
    assert ep.status_read(status) == ep.EP_FLAG_BAD_ROW
    assert (out[:16] == 5).all() and (out[-16:] == 5).all()


def test_overlapping_segments_that_fit_are_computed():
    """Every expert's weight gradient of the same rows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dy, x = ((torch.randint(-4, 5, (100, n), generator=g, device=DEV) * 0.5).to(torch.bfloat16) for n in (24, 40))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dw = ep.group_gemm_wgrad(dy, x, *segments(100), status=status)
    assert ep.status_read(status) == 0
    assert torch.equal(dw, (dy.double().T @ x.double()).float().expand(E, 24, 40))
