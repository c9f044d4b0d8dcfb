"""Windowed attention on the CPU: what the entry points refuse and workspace
sizes (nothing here launches a kernel)."""
import ctypes
import os

import pytest

from sparse_paged_kv_locks_gb300 import binding as B

FAKE = ctypes.c_void_p(1 << 12)   # never dereferenced: rejected first
ODD = ctypes.c_void_p((1 << 12) + 8)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = B.lib()
    before = lib.locks_kernel_launches()
    yield lib
    assert lib.locks_kernel_launches() == before   # nothing was launched


DECODE = ("q k v P table lens window sinks batch h_q h_kv pages o lse ws "
          "bytes stream").split()
CHUNK = ("q k v P table starts lens n window sinks batch h_q h_kv pages o lse "
         "ws bytes stream").split()
GOOD = dict(q=FAKE, k=FAKE, v=FAKE, P=10, table=FAKE, starts=FAKE, lens=FAKE,
            n=5, window=64, sinks=4, batch=2, h_q=8, h_kv=2, pages=16, o=FAKE,
            lse=FAKE, ws=FAKE, bytes=1 << 30, stream=None)


def both(L, **kw):
    a = {**GOOD, **kw}
    one = L.locks_window_decode(*[a[n] for n in DECODE])
    two = L.locks_window_attention(*[a[n] for n in CHUNK])
    assert one == two, (one, two)
    return one


@pytest.mark.parametrize("kw,want", [
    ({"window": 0}, 1), ({"window": -1}, 1), ({"sinks": -1}, 1),
    ({"batch": -1}, 1), ({"pages": 0}, 1), ({"P": 0}, 1), ({"h_q": 7}, 1),
    ({"h_kv": 0}, 1), ({"h_q": 34}, 2), ({"pages": 2 ** 26 + 1}, 2),
    ({"h_q": 65536, "h_kv": 65536}, 2),
    ({"q": None}, 1), ({"k": None}, 1), ({"v": None}, 1), ({"table": None}, 1),
    ({"lens": None}, 1), ({"o": None}, 1), ({"lse": None}, 1),
    ({"ws": None}, 1), ({"q": ODD}, 1), ({"k": ODD}, 1), ({"v": ODD}, 1),
    ({"o": ODD}, 1), ({"ws": ODD}, 1), ({"batch": 0, "q": None}, 0),
    ({"bytes": 255}, 3)])
def test_refusals(L, kw, want):
    assert both(L, **kw) == want


def test_refusals_of_one(L):
    def chunk(**kw):
        a = {**GOOD, **kw}
        return L.locks_window_attention(*[a[n] for n in CHUNK])

    def decode(**kw):
        a = {**GOOD, **kw}
        return L.locks_window_decode(*[a[n] for n in DECODE])

    assert chunk(starts=None) == 1 and chunk(n=-1) == 1
    assert chunk(n=0, q=None) == 0
    assert chunk(n=2 ** 28) == 2               # rows
    assert chunk(P=2 ** 26) == 2               # rows of the caches' maps
    assert decode(batch=41713) == 2
    # entries of all lists: 2 * 2^16 * (2^14 + ...) and a warp's run past them
    assert decode(batch=40000, window=2 ** 20, pages=2 ** 20) == 2
    # a window that says no more than the table does
    need = B.locks_window_workspace_size(2, 2, 8, 2, 16, 2 ** 31 - 1,
                                         2 ** 31 - 1)
    most = B.EVERY_TOKEN
    assert decode(window=most, sinks=most, bytes=need - 1) == 3


def size(*a):
    return B.locks_window_workspace_size(*a)


def test_size_refusals(L):
    out = ctypes.c_size_t(0)
    ok = (5, 2, 8, 2, 16, 64, 4)
    assert L.locks_window_workspace_size(*ok, ctypes.byref(out)) == 0
    assert L.locks_window_workspace_size(*ok, None) == 1
    for i, v, want in ((0, -1, 1), (1, -1, 1), (2, 7, 1), (2, 34, 2),
                       (3, 0, 1), (4, 0, 1), (4, 2 ** 26 + 1, 2), (5, 0, 1),
                       (6, -1, 1)):
        bad = list(ok)
        bad[i] = v
        assert L.locks_window_workspace_size(*bad, ctypes.byref(out)) == want


@pytest.mark.parametrize("h_kv,G", [(8, 4), (8, 8), (1, 16), (2, 1), (3, 5)])
def test_workspace_grows_with_every_size(L, h_kv, G):
    # a server allocates once, for its largest calls
    h_q = h_kv * G
    base = [300, 4, h_q, h_kv, 600, 2000, 40]
    steps = {0: [1, 2, 25, 26, 63, 64, 65, 300, 2000, 9000, 100000],
             1: [1, 2, 3, 9, 40, 200, 2000],
             4: [1, 7, 8, 9, 63, 600, 5000], 5: [1, 2, 100, 128, 129, 9000,
                                                 2 ** 31 - 1],
             6: [0, 1, 127, 128, 129, 5000, 2 ** 31 - 1]}
    for i, values in steps.items():
        for other in ({}, {0: 3}, {4: 9000}, {5: 2 ** 31 - 1}):
            a = list(base)
            for k, v in other.items():
                a[k] = v
            got = []
            for v in values:
                a[i] = v
                got.append(size(*a))
            assert got == sorted(got), (i, other)


def test_calls_fit_their_workspaces(L):
    """The call that finds its workspace too small by a byte is refused, for
    sizes on every side of the rules (the size itself is checked by tests that
    run the kernels)."""
    for n in (1, 4, 64, 65, 300, 5000):
        for batch in (1, 2, 16):
            for pages in (1, 9, 2000):
                for window in (1, 300, 2 ** 31 - 1):
                    need = size(n, batch, 8, 2, pages, window, 5)
                    a = {**GOOD, "n": n, "batch": batch, "pages": pages,
                         "window": window, "sinks": 5, "bytes": 200}
                    assert need >= 256
                    assert L.locks_window_attention(
                        *[a[x] for x in CHUNK]) == 3


def test_binding_refuses_cpu_tensors(L):
    import torch
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    i = torch.zeros(2, dtype=torch.int32)
    lse = torch.zeros(2, 8)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.locks_window_decode(q, kc, kc, t, i, 4, 0, q, lse, ws)
    with pytest.raises(ValueError):
        B.locks_window_attention(q, kc, kc, t, torch.zeros(3, dtype=torch.int32),
                                 i, 4, 0, q, lse, ws)


@pytest.mark.parametrize("window,sinks", [
    (2 ** 31, 0), (2 ** 32 + 5, 0), (16, 2 ** 32), (16, 2 ** 40 + 1),
    (-2 ** 32 + 16, 0)])
def test_binding_refuses_what_int32_does_not_hold(L, window, sinks):
    with pytest.raises(ValueError, match="EVERY_TOKEN"):
        B.locks_window_workspace_size(1, 1, 1, 1, 1, window, sinks)
    assert B.locks_window_workspace_size(1, 1, 1, 1, 1, B.EVERY_TOKEN,
                                         B.EVERY_TOKEN) > 0


def ranges(n, batch, h_kv, G, pages, window, sinks):
    """The number of ranges that a call cuts each unit's tiles into, stated
    apart from the library: the least estimate of rounds of units, each of its
    tiles, its start and end, and of joining."""
    tokens = 2 * (128 // G)
    window, sinks = min(window, 16 * pages), min(sinks, 16 * pages)
    tiles = min((min(tokens, n) + window + 126) // 128 + 1 +
                (sinks + 127) // 128, (16 * pages + 127) // 128)
    units = max(-(-n // tokens), batch) * h_kv
    rows = n * h_kv * G
    best, cost = 1, None
    for s in range(1, min(64, tiles) + 1):
        if s > 1 and rows * s > 65536:
            break
        c = -(-units * s // 152) * (-(-tiles // s) + 3.5)
        if s > 1:
            c += 3.0 + 1.2e-4 * (rows * s)
        if cost is None or c < cost:
            best, cost = s, c
    return best


def test_a_call_needs_no_more_than_the_size_reported(L):
    """Of one byte less than its own ranges' partials a call is refused, and
    that is within the size reported, for sizes on every side of the rules.
    (Where there is no GPU, so that a call which is not refused ends there.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls' pointers are not memory")
    seen = set()
    for n in (1, 4, 17, 64, 65, 300, 1365, 5000):
        for batch in (1, 2, 16, 130):
            for h_kv, G in ((8, 4), (1, 16), (2, 5)):
                for pages in (1, 9, 150, 2000, 30000):
                    for window, sinks in ((1, 0), (300, 5), (5000, 200),
                                          (2 ** 31 - 1, 0)):
                        s = ranges(n, batch, h_kv, G, pages, window, sinks)
                        seen.add(s)
                        rows = s * n * h_kv * G if s > 1 else 0
                        own = 256 + rows * 512 + -(-rows * 8 // 256) * 256
                        need = size(n, batch, h_kv * G, h_kv, pages, window,
                                    sinks)
                        assert own <= need
                        a = {**GOOD, "n": n, "batch": batch, "h_kv": h_kv,
                             "h_q": h_kv * G, "pages": pages,
                             "window": window, "sinks": sinks,
                             "bytes": own - 1}
                        assert L.locks_window_attention(
                            *[a[x] for x in CHUNK]) == 3, (a, s)
    assert len(seen) > 20
