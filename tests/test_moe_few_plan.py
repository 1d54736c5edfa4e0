"""The few-token layer's plan: what a block writes into its shared memory lies
inside what it asks for, whatever the route (no GPU needed: the arithmetic that
the kernels and their launcher share is compiled for the host)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_ep_layout_02_gb300", "csrc")

SHIM = r"""
#include "ep_few_plan.h"
extern "C" int group_limit(int T) { return ep::group_limit(T); }
extern "C" int group_count(int n, int limit) { return ep::group_count(n, limit); }
extern "C" int group_size(int n, int i, int limit) { return ep::group_size(n, i, limit); }
extern "C" void up_plan(int T, int H, int C, size_t shared, size_t* out) {
    const ep::UpPlan p = ep::up_plan(T, H, C, shared);
    const size_t v[] = {(size_t)p.rows, (size_t)p.stride, p.shared, p.scales, p.part, p.bytes};
    for (int i = 0; i < 6; ++i) out[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = str(d / "plan.cpp"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC,
                    "-I" + os.path.join(ROOT, "include"), src, "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.up_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p]

    def up_plan(T, H, C, shared):
        out = (ctypes.c_size_t * 6)()
        so.up_plan(T, H, C, shared, out)
        return dict(zip(("rows", "stride", "shared", "scales", "part", "bytes"), list(out)))
    so.plan_of = up_plan
    return so


def groups(plan, T, k, pairs_of_one):
    """Sizes of the groups that one expert's pairs make."""
    limit = plan.group_limit(T)
    n = plan.group_count(pairs_of_one, limit)
    return [plan.group_size(pairs_of_one, i, limit) for i in range(n)]


@pytest.mark.parametrize("T", list(range(1, 10)) + [33, 64])
@pytest.mark.parametrize("k", [1, 2, 8, 32])
def test_an_experts_pairs_make_whole_groups(plan, T, k):
    # a token may name one expert up to k times
    for n in range(1, T * k + 1):
        sizes = groups(plan, T, k, n)
        assert sum(sizes) == n and len(sizes) <= n
        assert all(1 <= s <= 8 for s in sizes)


@pytest.mark.parametrize("T", list(range(1, 10)) + [64])
@pytest.mark.parametrize("k", [1, 2, 8, 32])
@pytest.mark.parametrize("H", [128, 2048, 7168, 16384])
@pytest.mark.parametrize("C", [1, 2, 4])
def test_rows_and_scales_stay_in_their_places(plan, T, k, H, C):
    shared = 20488
    p = plan.plan_of(T, H, C, shared)
    most = max(s for n in range(1, T * k + 1) for s in groups(plan, T, k, n))  # rows that the cast writes
    assert (most - 1) * p["stride"] + H <= p["shared"]
    assert p["shared"] + shared <= p["scales"]
    assert p["scales"] + most * (H // 128) * 4 <= p["part"]
    assert p["part"] + (C - 1) * 8 * 2 * 32 * 16 <= p["bytes"]
    assert p["stride"] % 16 == 0 and p["shared"] % 16 == 0 and p["scales"] % 4 == 0 and p["part"] % 16 == 0
