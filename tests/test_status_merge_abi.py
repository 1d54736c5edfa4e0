"""Host-side argument checks of ep_status_merge (no GPU needed: every call is
refused before anything is enqueued)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from combine_ep_layout_02_gb300 import build as cuda_build
    cuda_build.build()
    from combine_ep_layout_02_gb300 import binding
    return binding.load()


def test_status_merge_argument_validation(lib):
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731  never dereferenced
    assert lib.ep_status_merge(None, at(0), None) == 1 and lib.ep_status_merge(at(0), None, None) == 1
    assert lib.ep_status_merge(at(2), at(0), None) == 2 and lib.ep_status_merge(at(0), at(1), None) == 2
