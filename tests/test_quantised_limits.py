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


def prefix_size(batch, h_q, h_kv, max_pages, pages):
    return B.locks_prefix_workspace_size(batch, h_q, h_kv, max_pages, pages)


@pytest.mark.parametrize("h_kv,G", [(8, 4), (8, 8), (1, 16), (2, 1), (3, 5)])
def test_prefix_workspace_grows_with_every_size(L, h_kv, G):
    # a server allocates once for its largest batch, prefix and tables and
    # serves fewer sequences and shorter prefixes from that
    h_q, top = h_kv * G, 9000
    for pages in (1, 12, 200, 1729, 1777, 8192):
        sizes = [prefix_size(b, h_q, h_kv, top, pages) for b in range(0, 400)]
        assert sizes == sorted(sizes)
    for batch in (2, 3, 32, 64, 110, 111, 300):
        sizes = [prefix_size(batch, h_q, h_kv, top, p) for p in range(0, 8200)]
        assert sizes == sorted(sizes)
        sizes = [prefix_size(batch, h_q, h_kv, n, 900)
                 for n in range(900, 6000, 37)]
        assert sizes == sorted(sizes)


def test_prefix_workspace_of_the_largest_serves_smaller(L):
    most = prefix_size(128, 32, 8, 9000, 8192)
    for batch in (1, 2, 31, 110, 111, 128):
        for pages in (0, 100, 1729, 1777, 8192):
            assert prefix_size(batch, 32, 8, 9000, pages) <= most
            # refused below its own size, by the call as well
            need = prefix_size(batch, 32, 8, 9000, pages)
            assert L.locks_prefix_decode(
                FAKE, FAKE, 10, FAKE, pages, FAKE, FAKE, batch, 32, 8, 9000,
                FAKE, FAKE, FAKE, need - 1, None) == 3
