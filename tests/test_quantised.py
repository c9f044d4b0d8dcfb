"""The quantised cache's format on the CPU: the oracle against closed forms
and an independent conversion, and the refusals of its entry points (nothing
here launches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import quantised_oracle as Q
from sparse_paged_kv_locks_gb300 import binding as B


# ---------------------------------------------------------------------------
# the format
# ---------------------------------------------------------------------------
def test_table_against_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes.to(torch.float64).numpy(), Q.TABLE)


def test_codes_against_torch():
    # torch converts to nearest even; its overflow differs, so inputs are
    # scaled rows
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 128)).astype(np.float32)
    x *= 2.0 ** rng.integers(-20, 20, (200, 1))
    x[:, ::7] *= 1e-3
    codes, e = Q.quantise_rows(x)
    scaled = torch.from_numpy(np.ldexp(x.astype(np.float64),
                                       -e[:, None]).astype(np.float32))
    assert scaled.abs().max() <= 448
    want = scaled.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(codes, want)


@pytest.mark.parametrize("x,e", [
    (448.0, 0), (np.nextafter(np.float32(448), np.float32(500)), 1),
    (224.0, -1), (225.0, 0), (0.0, -32), (1e-30, -32), (448.0 * 2.0 ** 31, 31),
    (3e38, 31), (np.inf, 31)])
def test_exponent_edges(x, e):
    assert Q.exponent(float(x)) == e


def test_error_bound_and_special_numbers():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 128)) * 2.0 ** rng.integers(-6, 7, (50, 128))
    codes, e = Q.quantise_rows(x)
    back = Q.TABLE[codes] * 2.0 ** e[:, None]
    # half a step: 2^-4 of a normal code, half the smallest code below
    bound = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e[:, None] - 10.0))
    assert (np.abs(back - x) <= bound).all()
    row = np.zeros((1, 128))
    row[0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    codes, e = Q.quantise_rows(row)
    assert e[0] == 31
    back = Q.TABLE[codes[0]] * 2.0 ** 31
    assert np.isnan(back[0]) and back[1] == 448 * 2.0 ** 31 == -back[2]
    row[0, 1:3] = 0.0   # a NaN leaves the row's scale to its numbers
    codes, e = Q.quantise_rows(row)
    assert e[0] == -8 and Q.TABLE[codes[0, 3]] * 2.0 ** -8 == 1.0
    assert np.isnan(Q.TABLE[codes[0, 0]])


def test_ties_go_to_even_codes():
    # 448 fixes the scale at 1; 9 = 8 + 1 is a code, 8.5 and 9.5 are ties
    row = np.zeros((1, 128))
    row[0, :5] = [448.0, 8.5, 9.5, -8.5, 2.0 ** -10]
    codes, e = Q.quantise_rows(row)
    got = Q.TABLE[codes[0, :5]]
    assert e[0] == 0
    np.testing.assert_array_equal(got, [448.0, 8.0, 10.0, -8.0, 0.0])


def test_places_are_a_permutation_without_bank_conflicts():
    place = np.array([[Q.byte_of(s, d) for d in range(128)]
                      for s in range(16)])
    assert sorted(place.reshape(-1)) == list(range(2048))
    group = place[:, ::16] // 16 % 8     # [slot][c]: 16-byte bank group
    for r in (0, 8):
        # keys: rows 2i, 2i + 1, groups 4j .. 4j + 3 in one pass
        for i in range(4):
            for j in range(2):
                at = {group[r + 2 * i + a, 4 * j + t] for a in range(2)
                      for t in range(4)}
                assert len(at) == 8
        # values: rows 2t (or 2t + 1), groups 2i, 2i + 1
        for i in range(4):
            for odd in range(2):
                at = {group[r + 2 * t + odd, 2 * i + a] for a in range(2)
                      for t in range(4)}
                assert len(at) == 8


def test_oracle_write_read_and_attention():
    rng = np.random.default_rng(2)
    cache = np.zeros((5, 2, Q.RECORD), np.uint8)
    table = np.array([[3, 0], [1, 4]], np.int32)
    n = 23
    k = rng.standard_normal((n, 2, 128))
    v = rng.standard_normal((n, 2, 128))
    Q.write(cache, k, v, [1] * n, list(range(n)), table)
    K, V = Q.tokens(cache, table[1], 1, range(2), n)
    codes, e = Q.quantise_rows(k[:, 1])
    np.testing.assert_array_equal(K, Q.TABLE[codes] * 2.0 ** e[:, None])
    assert np.abs(V - v[:, 1]).max() <= 2.0 ** -4 * np.abs(v).max()
    assert not cache[[0, 2, 3]].any()     # other pages untouched
    q = rng.standard_normal((2, 4, 128))
    o, lse, _ = Q.decode(q, cache, table, [0, n])
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    # one head by hand
    w = np.exp(q[1, 3] @ K.T / np.sqrt(128))
    np.testing.assert_allclose(o[1, 3], w @ V / w.sum(), rtol=1e-12)
    np.testing.assert_allclose(lse[1, 3], np.log(w.sum()), rtol=1e-12)
    # a shared prefix takes the place of the table's first entries
    other = np.array([[2, 0], [2, 4]], np.int32)
    o2, lse2, _ = Q.decode(q, cache, other, [0, n], prefix=[1])
    np.testing.assert_array_equal(o2, o)
    np.testing.assert_array_equal(lse2, lse)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
FAKE = ctypes.c_void_p(1 << 12)   # never dereferenced: rejected first
ODD = ctypes.c_void_p((1 << 12) + 8)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = B.lib()
    before = lib.locks_kernel_launches()
    yield lib
    assert lib.locks_kernel_launches() == before   # nothing was launched


def changed(args, **at):
    out = list(args)
    for i, v in at.items():
        out[int(i[1:])] = v
    return out


def test_quantise_refusals(L):
    ok = [FAKE, FAKE, 0, 1024, 128, 1024, 128, FAKE, FAKE, 3, FAKE, 10, 8,
          FAKE, 2, 16, None, None]
    f = L.locks_quantise_kv
    for i in (0, 1, 7, 8, 10, 13):                 # null pointers
        assert f(*changed(ok, **{f"a{i}": None})) == 1
    for i in (0, 1, 10):                           # misaligned
        assert f(*changed(ok, **{f"a{i}": ODD})) == 1
    for i in (3, 4, 5, 6):                         # strides off 16 bytes
        assert f(*changed(ok, **{f"a{i}": 1028})) == 1
    assert f(*changed(ok, a2=2, a3=1022)) == 1     # fp32: 4 elements
    for i, v in ((2, 3), (2, -1), (9, -1), (11, 0), (12, 0), (14, 0),
                 (15, 0)):
        assert f(*changed(ok, **{f"a{i}": v})) == 1
    assert f(*changed(ok, a9=1 << 30, a12=2)) == 2
    assert f(*changed(ok, a15=1 << 28)) == 2
    assert f(*changed(ok, a9=0, a0=None)) == 0     # nothing to write


def test_dequantise_refusals(L):
    ok = [FAKE, 10, 8, FAKE, 2, 16, FAKE, FAKE, 3, None, 0, FAKE, FAKE, None,
          None]
    f = L.locks_dequantise_kv
    for i in (0, 3, 6, 7):
        assert f(*changed(ok, **{f"a{i}": None})) == 1
    assert f(*changed(ok, a11=None, a12=None)) == 1
    for i in (0, 11, 12):
        assert f(*changed(ok, **{f"a{i}": ODD})) == 1
    for i, v in ((10, 3), (8, -1), (1, 0), (2, 0), (4, 0), (5, 0)):
        assert f(*changed(ok, **{f"a{i}": v})) == 1
    assert f(*changed(ok, a8=1 << 30, a2=2)) == 2
    assert f(*changed(ok, a8=0, a0=None)) == 0


def test_decode_refusals(L):
    ok = [FAKE, FAKE, 10, FAKE, FAKE, FAKE, 4, 2, 8, 2, 16, FAKE, FAKE, FAKE,
          1 << 30, None]
    f = L.locks_quantised_decode
    for i in (0, 1, 3, 4, 11, 12, 13):
        assert f(*changed(ok, **{f"a{i}": None})) == 1
    for i in (0, 1, 11, 13):
        assert f(*changed(ok, **{f"a{i}": ODD})) == 1
    for i, v in ((2, 0), (6, 0), (7, -1), (8, 7), (9, 0), (10, 0)):
        assert f(*changed(ok, **{f"a{i}": v})) == 1
    assert f(*changed(ok, a8=34)) == 2             # 17 heads to a KV head
    assert f(*changed(ok, a7=41089)) == 2
    assert f(*changed(ok, a7=41088, a14=64)) == 3
    assert f(*changed(ok, a6=1 << 30)) == 2        # positions past 2^31
    need = B.locks_workspace_size(2, 8, 2, 16, 4)
    assert f(*changed(ok, a14=64)) == 3 and need > 64
    assert f(*changed(ok, a7=0, a0=None)) == 0


def test_prefix_refusals(L):
    ok = [FAKE, FAKE, 10, FAKE, 5, FAKE, FAKE, 2, 8, 2, 16, FAKE, FAKE, FAKE,
          1 << 30, None]
    f = L.locks_prefix_decode
    for i in (0, 1, 3, 5, 6, 11, 12, 13):
        assert f(*changed(ok, **{f"a{i}": None})) == 1
    for i in (0, 1, 11, 13):
        assert f(*changed(ok, **{f"a{i}": ODD})) == 1
    for i, v in ((2, 0), (4, -1), (4, 17), (7, -1), (8, 7), (9, 0), (10, 0)):
        assert f(*changed(ok, **{f"a{i}": v})) == 1
    assert f(*changed(ok, a8=34)) == 2
    need = B.locks_prefix_workspace_size(2, 8, 2, 16, 5)
    assert f(*changed(ok, a14=need - 1)) == 3
    assert f(*changed(ok, a7=0, a0=None)) == 0
    out = ctypes.c_size_t(0)
    g = L.locks_prefix_workspace_size
    assert g(2, 8, 2, 16, 17, ctypes.byref(out)) == 1
    assert g(2, 34, 2, 16, 4, ctypes.byref(out)) == 2
    assert g(2, 8, 2, 16, 4, None) == 1


def test_workspace_covers_both_decodes(L):
    # the workspace of locks_workspace_size is never too small for the
    # quantised decode, whichever region decides its size
    f = L.locks_quantised_decode
    for batch, h_q, h_kv, pages, k in ((1, 16, 1, 1, 1), (3, 8, 2, 4, 300),
                                       (32, 32, 8, 64, 64)):
        need = B.locks_workspace_size(batch, h_q, h_kv, pages, k)
        args = [FAKE, FAKE, 10, FAKE, FAKE, FAKE, k, batch, h_q, h_kv, pages,
                FAKE, FAKE, FAKE, need, None]
        assert f(*changed(args, a14=256)) == 3
        rows = (batch * h_kv + min(8192, batch * h_kv * k)) * h_q // h_kv
        assert need >= 256 + 4 * (batch + 2) + rows * (512 + 8)


def test_binding_refusals(L):
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    ids = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    cache = torch.zeros(4, 2, 4128, dtype=torch.uint8)
    with pytest.raises(ValueError):                # CPU tensors
        B.locks_quantise_kv(rows, rows, ids, ids, table, cache)
    with pytest.raises(TypeError):
        B.locks_quantise_kv(rows, rows, ids, ids, table, cache.int())
    with pytest.raises(ValueError):
        B.locks_dequantise_kv(cache, table, ids, ids, None, None)
    with pytest.raises(ValueError):
        B.locks_quantised_decode(rows, cache, table, ids, None, 4, rows,
                                 torch.zeros(3, 2), cache.view(-1))
