"""Rotary positions on the CPU: the fractions of a turn, and what the entry
points refuse (nothing here launches a kernel)."""
import ctypes
import os
from fractions import Fraction

import pytest

from sparse_paged_kv_locks_gb300 import binding as B

FAKE = ctypes.c_void_p(1 << 12)   # never dereferenced: rejected first
ODD = ctypes.c_void_p((1 << 12) + 8)
# 2 pi to 60 digits
TWO_PI = Fraction(
    "6.28318530717958647692528676655900576839433879875021164194988")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = B.lib()
    before = lib.locks_kernel_launches()
    yield lib
    assert lib.locks_kernel_launches() == before   # nothing was launched


@pytest.mark.parametrize("f", [1.0, 0.1, 500000.0 ** (-63 / 64), 1e-9, 6.25,
                               1048576.0, -1.0, -1e-3, -1e-30, 0.0, 1e-300])
def test_turns_are_good_to_their_last_bits(L, f):
    r = B.Rotation([f] * 8)
    want = Fraction(f) / TWO_PI * 2 ** 64
    off = (r.struct.turns[0] - want) % 2 ** 64
    # the fraction is rounded once (half a unit); a product whose size is
    # above 2^-53 of a turn has its double-double's error too, 2^-104 of it
    assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 1000) + \
        abs(Fraction(f)) * Fraction(1, 2 ** 40)


def test_struct_holds_what_was_given(L):
    r = B.Rotation.of_base(10000.0, 96, sections=(8, 20, 20), pairs=True,
                           amplitude=1.25)
    s = r.struct
    assert (s.dim, s.pairs, s.n_axes, s.amplitude) == (96, 1, 3, 1.25)
    assert list(s.axes) == [0] * 8 + [1] * 20 + [2] * 20 + [0] * 16
    assert list(s.turns[48:]) == [0] * 16
    assert r.n_axes == 3 and B.Rotation([1.0] * 8).n_axes == 1
    assert ctypes.sizeof(s) == 64 * 9 + 16


@pytest.mark.parametrize("kw", [
    {"frequencies": []}, {"frequencies": [1.0] * 7},
    {"frequencies": [1.0] * 72}, {"frequencies": [float("nan")] * 8},
    {"frequencies": [float("inf")] * 8}, {"frequencies": [2.0 ** 21] * 8},
    {"frequencies": [1.0] * 8, "axes": [0] * 7 + [4]},
    {"frequencies": [1.0] * 8, "axes": [0] * 7 + [-1]},
    {"frequencies": [1.0] * 8, "axes": [0] * 7 + [2], "n_axes": 2},
    {"frequencies": [1.0] * 8, "n_axes": 0},
    {"frequencies": [1.0] * 8, "amplitude": float("inf")}])
def test_rotation_refusals(L, kw):
    with pytest.raises(B.LocksError):
        B.Rotation(**kw)
    with pytest.raises(ValueError):
        B.Rotation([1.0] * 8, axes=[0] * 9)


NAMES = ("q k v type qt qh kt kh vt vh rot rotary seq pos n h_q q_out cache "
         "P h_kv table batch pages status").split()
GOOD = dict(q=FAKE, k=FAKE, v=FAKE, type=0, qt=1024, qh=128, kt=256, kh=128,
            vt=256, vh=128, rotary=None, seq=FAKE, pos=FAKE, n=3, h_q=8,
            q_out=FAKE, cache=FAKE, P=10, h_kv=2, table=FAKE, batch=2,
            pages=16, status=None)


def rotate(L, **kw):
    a = {**GOOD, "rot": B.Rotation([1.0] * 64)._at, **kw}
    args = [a[n] for n in NAMES]
    one = L.locks_rotate_quantise_kv(*args, None)
    at = NAMES.index("cache") + 1
    two = L.locks_rotate_kv(*args[:at], FAKE, *args[at:], None)
    assert one == two, (one, two)
    return one


@pytest.mark.parametrize("kw,want", [
    ({"rot": None}, 1), ({"type": 3}, 1), ({"n": -1}, 1), ({"h_kv": 0}, 1),
    ({"batch": 0}, 1), ({"pages": 0}, 1), ({"P": 0}, 1), ({"h_q": 0}, 1),
    ({"k": None}, 1), ({"v": None}, 1), ({"seq": None}, 1),
    ({"pos": None}, 1), ({"cache": None}, 1), ({"table": None}, 1),
    ({"q_out": None}, 1), ({"q": ODD}, 1), ({"k": ODD}, 1), ({"v": ODD}, 1),
    ({"q_out": ODD}, 1), ({"cache": ODD}, 1), ({"qt": 1028}, 1),
    ({"kh": 132}, 1), ({"vt": 4}, 1), ({"type": 2, "vt": 130}, 1),
    ({"n": 2 ** 31 - 1}, 2), ({"pages": 2 ** 27}, 2),
    ({"n": (2 ** 31 - 1) // 12 + 1}, 2), ({"n": 0, "k": None}, 0)])
def test_rotate_refusals(L, kw, want):
    assert rotate(L, **kw) == want


def test_a_struct_that_was_not_filled_is_refused(L):
    for field, value in (("dim", 8), ("dim", 144), ("dim", 24), ("pairs", 2),
                         ("n_axes", 0), ("n_axes", 5)):
        r = B.Rotation([1.0] * 8)
        setattr(r.struct, field, value)
        assert rotate(L, rot=r._at) == 1
    r = B.Rotation([1.0] * 8)
    r.struct.axes[3] = 1
    assert rotate(L, rot=r._at) == 1


def test_append_refusals(L):
    rot = B.Rotation([1.0] * 64)._at
    good = [FAKE, FAKE, FAKE, rot, None, 8, FAKE, FAKE, FAKE, 10, 2, FAKE, 1,
            16, FAKE, FAKE, None, 0, None, None]

    def call(**at):
        args = list(good)
        for i, v in at.items():
            args[int(i[1:])] = v
        return L.locks_append_rotated_kv(*args)

    for i in (0, 1, 2, 3, 6, 7, 8, 11, 14, 15):
        assert call(**{f"_{i}": None}) == 1, i
    assert call(_5=7) == 1 and call(_9=0) == 1 and call(_13=0) == 1
    assert call(_12=-1) == 1 and call(_17=2) == 1
    assert call(_0=ODD) == 1 and call(_6=ODD) == 1
    assert call(_5=34, _10=17) == 2
    assert call(_12=0) == 0


def test_binding_refuses_cpu_tensors(L):
    import torch
    rot = B.Rotation([1.0] * 64)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.locks_rotate_kv(None, k, k, rot, i, i, t, None, kc, kc)
    with pytest.raises(ValueError):
        B.locks_rotate_quantise_kv(None, k, k, rot, i, i, t, None,
                                   torch.zeros(4, 2, 4128, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.locks_append_rotated_kv(k, k, k, rot, k, kc, kc, t, i,
                                  torch.zeros(1, 2, 4, 832,
                                              dtype=torch.uint8))


def test_positions_are_checked_by_their_shape(L):
    """[n][n_axes], which has as many numbers as [n_axes][n], is refused.  (On
    the CPU, whose tensors are on GPU -1.)"""
    import torch
    three = B.Rotation([1.0] * 9 + [0.5] * 7, axes=[0] * 4 + [1] * 6 + [2] * 6)
    one = B.Rotation([1.0] * 8)

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    for rot, t in ((three, ints(3, 5)), (one, ints(1, 5)), (one, ints(5))):
        B._req_rotary(-1, t, rot, 5, "n")
        B._req_turning(-1, rot, t, True, 5)
    for rot, t in ((three, ints(5, 3)), (three, ints(15)), (one, ints(5, 1)),
                   (three, ints(1, 5)), (one, ints(3, 5)), (one, ints(4)),
                   (three, ints(5, 3).t()), (one, ints(1, 10)[:, ::2])):
        with pytest.raises(ValueError):
            B._req_rotary(-1, t, rot, 5, "n")
        with pytest.raises(ValueError):
            B._req_turning(-1, rot, t, True, 5)
    with pytest.raises(TypeError):
        B._req_turning(-1, three, ints(3, 5).long(), True, 5)


def test_a_decoder_checks_its_rotation_at_once(L):
    rot = B.Rotation([1.0] * 8)
    B._req_turning(-1, None, None, False, 5)
    B._req_turning(-1, rot, None, True, 5)
    with pytest.raises(TypeError):
        B._req_turning(-1, [1.0] * 8, None, True, 5)
    with pytest.raises(ValueError):
        B._req_turning(-1, rot, None, False, 5)


def test_append_refuses_rows_that_it_cannot_load(L):
    """Eight bytes a lane of keys, values and caches, sixteen of records, with
    a rotation and without."""
    off4, off8 = ctypes.c_void_p((1 << 12) + 4), ODD
    rot = B.Rotation([1.0] * 64)._at
    turned = [FAKE, FAKE, FAKE, rot, None, 8, FAKE, FAKE, FAKE, 10, 2, FAKE,
              0, 16, FAKE, FAKE, None, 0, None, None]
    plain = [FAKE, FAKE, FAKE, FAKE, 10, 2, FAKE, 0, 16, FAKE, FAKE, None, 0,
             None, None]
    for call, good, rows, batch, records in (
            (L.locks_append_rotated_kv, turned, (1, 2, 7, 8), 12, 15),
            (L.locks_append_kv_ex, plain, (0, 1, 2, 3), 7, 10)):
        assert call(*good) == 0            # a batch of none
        for i, bad in [(i, off4) for i in rows] + [(records, off8)]:
            args = list(good)
            args[batch], args[i] = 1, bad
            assert call(*args) == 1, i
