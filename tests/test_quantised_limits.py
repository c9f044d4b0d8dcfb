"""Limits of the quantised cache's entry points on the CPU: sizes whose index
arithmetic would pass 32 bits, and workspace sizes (nothing here launches a
kernel)."""
import ctypes
import os

import pytest

from sparse_paged_kv_locks_gb300 import binding as B

FAKE = ctypes.c_void_p(1 << 12)   # never dereferenced: rejected first


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = B.lib()
    before = lib.locks_kernel_launches()
    yield lib
    assert lib.locks_kernel_launches() == before   # nothing was launched


@pytest.mark.parametrize("batch,h_kv,most", [(1, 1, 2 ** 31 - 2 ** 16),
                                             (2, 8, 2 ** 27 - 2 ** 12)])
def test_list_entries_leave_room_for_a_window(L, batch, h_kv, most):
    # positions run up to a run and a window past the last list entry; with a
    # workspace that is too small nothing is launched either way
    for k, want in ((most, 3), (most + 1, 2), ((2 ** 31 - 1) // (batch * h_kv),
                                               2)):
        assert L.locks_quantised_decode(
            FAKE, FAKE, 10, FAKE, FAKE, FAKE, k, batch, h_kv, h_kv, 16, FAKE,
            FAKE, FAKE, 64, None) == want
    # every page of tables that long
    pages = 2 ** 27 - 1
    for batch, want in ((15, 3), (16, 2)):
        assert L.locks_prefix_decode(
            FAKE, FAKE, 10, FAKE, 5, FAKE, FAKE, batch, 1, 1, pages, FAKE,
            FAKE, FAKE, 64, None) == want
