"""GPU parity of the quantised KV cache operators against the float64 oracle.

Tolerances, derived from the number formats:
  * written bytes and numbers read back as bf16 or fp32: equal; read back as
    fp16: the fp16 rounding of the oracle's number, equal
  * o: rounded to bf16 once (half a step, 2^-8 of the value); weights rounded
    to fp16 (2^-11 of each term sum p |v|); fp32 accumulation, exponentials
    of 2^-22 and scores off by dx below (2^-13 + 2 dx of the same sum)
  * lse: fp32 scores with dx <= 2^-17 * max_t sum_d |q_d k_td| / sqrt(128)
    (128 products, 2^-24 each), plus 2^-20 of the lse itself
A query element 2^-22 below its head's largest loses bits in fp16: an error
of 2^-25 of the largest times |k|, far inside dx.
"""
import math

import numpy as np
import pytest
import torch

from oracle import locks_oracle as O
from oracle import quantised_oracle as Q
from sparse_paged_kv_locks_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# writing
# ---------------------------------------------------------------------------
def hard_rows(rng, n, h, dtype):
    """Rows over the type's range: ordinary, zero, tiny, huge, with NaN and
    infinities, and numbers on and beside code borders."""
    x = rng.standard_normal((n, h, 128)) * \
        2.0 ** rng.integers(-12, 12, (n, h, 1))
    kind = rng.integers(0, 8, (n, h))
    x[kind == 0] = 0.0
    x[kind == 1] *= 2.0 ** -30
    x[kind == 2] *= 2.0 ** (8 if dtype is torch.float16 else 40)
    x[kind == 3, 5] = np.nan
    x[kind == 4, 7] = -np.inf
    x[kind == 4, 9] = np.inf
    grid = np.concatenate([Q.TABLE[:127], (Q.TABLE[:126] + Q.TABLE[1:127]) / 2])
    x[kind == 5] = rng.choice(grid, (int((kind == 5).sum()), 128))
    x[kind == 6] = np.where(rng.random((int((kind == 6).sum()), 128)) < 0.02,
                            448.0, 1e-3)
    return torch.from_numpy(x).to(dtype)


def as_bytes_with_one_nan(rec):
    """Codes with every NaN code as 0x7f."""
    out = rec.copy()
    codes = out[..., :4096]
    codes[(codes & 0x7F) == 0x7F] = 0x7F
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16,
                                   torch.float32])
@pytest.mark.parametrize("h_kv,lens", [(1, [1]), (2, [16]), (3, [5, 0, 33]),
                                       (8, [17, 1])])
def test_write_matches_oracle(dtype, h_kv, lens):
    rng = np.random.default_rng(h_kv + len(lens))
    n, batch, max_pages = sum(lens), len(lens), 4
    table = rng.permutation(batch * max_pages + 2)[:batch * max_pages] \
        .reshape(batch, max_pages).astype(np.int32)
    seq = np.concatenate([np.full(m, b) for b, m in enumerate(lens)])
    past = rng.integers(0, 30, batch)
    pos = np.concatenate([past[b] + np.arange(m)
                          for b, m in enumerate(lens)]).astype(np.int64)
    k, v = hard_rows(rng, n, h_kv, dtype), hard_rows(rng, n, h_kv, dtype)
    start = rng.integers(0, 256, (batch * max_pages + 2, h_kv, Q.RECORD)) \
        .astype(np.uint8)
    want = start.copy()
    Q.write(want, k.double().numpy(), v.double().numpy(), seq, pos, table)
    cache = torch.from_numpy(start).to(DEV)
    st = word()
    B.locks_quantise_kv(k.to(DEV), v.to(DEV), i32(seq), i32(pos), i32(table),
                        cache, status=st)
    assert int(st) == 0
    np.testing.assert_array_equal(as_bytes_with_one_nan(cache.cpu().numpy()),
                                  as_bytes_with_one_nan(want))


@pytest.mark.parametrize("order", ["fused", "head major", "two tensors"])
def test_write_takes_strided_rows(order):
    rng = np.random.default_rng(3)
    n, h = 37, 4
    table = np.arange(3, dtype=np.int32)[None]
    if order == "fused":
        qkv = torch.from_numpy(rng.standard_normal((n, 16 + 2 * h, 128))) \
            .to(DEV, torch.bfloat16)
        k, v = qkv[:, 16:16 + h], qkv[:, 16 + h:]
    elif order == "head major":
        k, v = (torch.from_numpy(rng.standard_normal((h, n, 128)))
                .to(DEV, torch.bfloat16).transpose(0, 1) for _ in range(2))
    else:
        k = torch.from_numpy(rng.standard_normal((n, h, 128))) \
            .to(DEV, torch.bfloat16)
        v = torch.from_numpy(rng.standard_normal((n, h + 3, 128))) \
            .to(DEV, torch.bfloat16)[:, 1:1 + h]
    cache = B.new_quantised_cache(3, h, DEV)
    B.locks_quantise_kv(k, v, i32([0] * n), i32(range(n)), i32(table), cache)
    want = np.zeros((3, h, Q.RECORD), np.uint8)
    Q.write(want, k.double().cpu().numpy(), v.double().cpu().numpy(),
            [0] * n, range(n), table)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_write_skips_padding_and_reports_bad_tokens():
    rng = np.random.default_rng(4)
    table = np.array([[0, 1], [2, 9]], np.int32)   # 9 is outside the cache
    seq = np.array([0, -1, 2, 0, 0, 1, 1], np.int32)
    pos = np.array([3, 0, 0, -1, 32, 20, 2], np.int32)
    k = torch.from_numpy(rng.standard_normal((7, 2, 128))).to(torch.bfloat16)
    cache = B.new_quantised_cache(3, 2, DEV)
    want = cache.cpu().numpy()
    good = [0, 6]
    kn = k.double().numpy()[good]
    Q.write(want, kn, kn, seq[good], pos[good], table)
    kd = k.to(DEV)
    st = word()
    B.locks_quantise_kv(kd, kd, i32(seq), i32(pos), i32(table), cache,
                        status=st)
    assert int(st) == B.DEV_BAD_PAIR | B.DEV_BAD_PAGE_ID
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    st = word()                                    # padding alone is no error
    B.locks_quantise_kv(kd, kd, i32([-1] * 7), i32(pos), i32(table), cache,
                        status=st)
    assert int(st) == 0
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# caches of plain numbers, with rubbish wherever nothing may be read
# ---------------------------------------------------------------------------
def records(rng, P, h_kv, spread=2, centre=-9):
    """Random records: any finite codes, scales around 2^centre."""
    rec = rng.integers(0, 256, (P, h_kv, Q.RECORD)).astype(np.uint8)
    codes = rec[..., :4096]
    codes[(codes & 0x7F) == 0x7F] = 0x10
    rec[..., 4096:] = 127 + centre + rng.integers(-spread, spread + 1,
                                                  rec[..., 4096:].shape)
    return rec


def poison_past_ends(rec, table, lens):
    """NaN codes and absurd scales in the slots past each sequence's end."""
    for b, L in enumerate(lens):
        if L % 16:
            r = rec[table[b, L // 16]]
            for s in range(L % 16, 16):
                for part in (0, 1):
                    r[:, 2048 * part + Q._PLACE[s]] = 0x7F
                    r[:, 4096 + 16 * part + s] = 255


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16,
                                   torch.float32])
@pytest.mark.parametrize("h_kv,n", [(1, 1), (3, 7), (8, 16)])
def test_read_matches_oracle(dtype, h_kv, n):
    rng = np.random.default_rng(n)
    batch, max_pages = 2, 9
    table = rng.permutation(18).reshape(2, 9).astype(np.int32)
    rec = records(rng, 18, h_kv, spread=12, centre=-1)
    seq, pg = rng.integers(0, batch, n), rng.integers(0, max_pages, n)
    K, V = Q.read(rec[table[seq, pg]])
    out = [torch.full((n, h_kv, 16, 128), 7.0, dtype=dtype, device=DEV)
           for _ in range(2)]
    st = word()
    cache = torch.from_numpy(rec).to(DEV)
    B.locks_dequantise_kv(cache, i32(table), i32(seq), i32(pg), *out,
                          status=st)
    assert int(st) == 0
    for got, want in zip(out, (K, V)):
        np.testing.assert_array_equal(
            got.double().cpu().numpy(),
            torch.from_numpy(want).to(dtype).double().numpy())
        if dtype is not torch.float16:
            np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    # one of the two alone
    alone = torch.empty_like(out[1])
    B.locks_dequantise_kv(cache, i32(table), i32(seq), i32(pg), None, alone)
    assert torch.equal(alone, out[1])


def test_read_stops_at_lengths_and_reports_bad_pairs():
    rng = np.random.default_rng(6)
    lens = [37, 0, 16]
    table = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 99]], np.int32)
    rec = records(rng, 8, 2)
    poison_past_ends(rec, table, lens)
    seq = np.array([0, 0, 1, 2, 2, 3, 0], np.int32)
    pg = np.array([1, 2, 0, 0, 2, 0, 3], np.int32)
    k = torch.full((7, 2, 16, 128), 7.0, device=DEV)
    v = torch.full((7, 2, 16, 128), 7.0, device=DEV)
    st = word()
    B.locks_dequantise_kv(torch.from_numpy(rec).to(DEV), i32(table), i32(seq),
                          i32(pg), k, v, seq_lens=i32(lens), status=st)
    assert int(st) == B.DEV_BAD_PAIR | B.DEV_BAD_PAGE_ID
    K, V = Q.read(rec[np.array([1, 2, 3, 6, 0, 0, 0])])
    for got, want in ((k, K), (v, V)):
        want = np.where(np.isnan(want), 0.0, want)
        want[1, :, 5:] = 0.0
        want[2] = 0.0
        want[4:] = 0.0
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    st = word()
    B.locks_dequantise_kv(torch.from_numpy(rec).to(DEV), i32(table), i32(seq),
                          i32(pg), k, v, seq_lens=i32([37, -1, 49]),
                          status=st)
    assert int(st) & B.DEV_BAD_SEQ_LEN


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check(got_o, got_lse, q, rec, want, below=0.0):
    """`below`: what weights too small for fp16 may add up to (where one
    token takes nearly all of a row, dims in which its value is zero)."""
    o, lse, mass = want
    got_o = got_o.double().cpu().numpy()
    got_lse = got_lse.double().cpu().numpy()
    empty = np.isneginf(lse)
    np.testing.assert_array_equal(np.isneginf(got_lse), empty)
    assert (got_o[empty] == 0).all()
    # largest key row by magnitude bounds the products of a score
    K, _ = Q.read(rec)
    kmax = np.nanmax(np.where(np.isfinite(K) & (np.abs(K) < 1e30),
                              np.abs(K), 0.0))
    dx = 2.0 ** -17 * np.abs(q).sum(-1) * kmax / math.sqrt(128)
    tol = 2.0 ** -8 * np.abs(o) + \
        (2.0 ** -11 + 2.0 ** -13 + 2 * dx[..., None]) * mass
    bad = np.abs(got_o - o) > tol + 1e-30 + below
    assert not bad.any(), (np.argwhere(bad)[:5], got_o[bad][:5], o[bad][:5])
    ltol = dx + 2.0 ** -20 * np.abs(np.where(empty, 0, lse)) + 2.0 ** -20
    assert (np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, lse))
            <= ltol).all()


def queries(rng, batch, h_q, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal((batch, h_q, 128))) \
        .to(torch.bfloat16)


def selection(rng, lens, h_kv, k):
    """Ascending lists with sink and recent page and -1 where short."""
    idx = np.full((len(lens), h_kv, k), -1, np.int32)
    for b, L in enumerate(lens):
        n = -(-L // 16)
        for h in range(h_kv):
            if n <= k:
                pages = np.arange(n)
            else:
                mid = rng.permutation(np.arange(1, n - 1))[:k - 2]
                pages = np.sort(np.concatenate([[0], mid, [n - 1]]))[:k]
            idx[b, h, :len(pages)] = pages
    return idx


def run_decode(q, rec, table, lens, idx=None, k=0, stream=None):
    batch, h_q, _ = q.shape
    h_kv, max_pages = rec.shape[1], table.shape[1]
    k = k or max_pages
    o = torch.full((batch, h_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((batch, h_q), 7.0, device=DEV)
    ws = B.new_workspace(batch, h_q, h_kv, max_pages, k, DEV)
    args = (q.to(DEV), torch.from_numpy(rec).to(DEV), i32(table), i32(lens),
            None if idx is None else i32(idx), k, o, lse, ws)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    B.locks_quantised_decode(*args, stream=stream)
    torch.cuda.synchronize()
    return o, lse, B.locks_read_status(ws)


def case(rng, lens, h_kv, spread=2, centre=-9, room=2):
    batch = len(lens)
    max_pages = max(1, -(-max(lens) // 16)) + room
    P = batch * max_pages + 3
    table = rng.permutation(P)[:batch * max_pages].reshape(
        batch, max_pages).astype(np.int32)
    rec = records(rng, P, h_kv, spread, centre)
    poison_past_ends(rec, table, lens)
    return rec, table


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("lens,h_kv", [([1], 1), ([0, 15, 16, 17], 2),
                                       ([333, 1, 0, 90, 31], 3)])
def test_dense_decode(G, lens, h_kv):
    rng = np.random.default_rng(G)
    rec, table = case(rng, lens, h_kv)
    q = queries(rng, len(lens), G * h_kv)
    o, lse, st = run_decode(q, rec, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens))


@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("lens,h_kv,room", [
    ([9000, 100, 0, 16], 1, 0), ([333, 1, 0, 90, 31], 3, 700),
    ([0, 0], 2, 900), ([4000, 3990, 17], 2, 600)])
def test_dense_decode_over_long_tables(G, lens, h_kv, room):
    # tables too long for one unit to a CTA: runs over all lists, units that
    # span many runs, runs that span many units, units of no pages
    rng = np.random.default_rng(G + room)
    rec, table = case(rng, lens, h_kv, room=room)
    q = queries(rng, len(lens), G * h_kv)
    o, lse, st = run_decode(q, rec, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens))


def test_dense_decode_of_many_units():
    rng = np.random.default_rng(21)
    lens = [int(x) for x in rng.integers(0, 1100, 90)]
    for room in (0, 300):          # one CTA to a unit, and runs
        rec, table = case(rng, lens, 2, room=room)
        q = queries(rng, 90, 10)
        o, lse, st = run_decode(q, rec, table, lens)
        assert st == 0
        qn = q.double().numpy()
        check(o, lse, qn, rec, Q.decode(qn, rec, table, lens))


@pytest.mark.parametrize("G", [1, 4, 5, 8, 16])
@pytest.mark.parametrize("lens,h_kv,k", [
    ([700], 1, 2), ([40, 0, 900, 17], 2, 5),      # few entries: split runs
    ([640, 320], 2, 16), ([2000, 1500], 2, 64),   # clusters of several sizes
    ([513], 1, 40), ([300, 77, 16], 3, 12)])
def test_listed_decode(G, lens, h_kv, k):
    rng = np.random.default_rng(G + k)
    rec, table = case(rng, lens, h_kv)
    q = queries(rng, len(lens), G * h_kv)
    idx = selection(rng, lens, h_kv, k)
    o, lse, st = run_decode(q, rec, table, lens, idx, k)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, idx))


@pytest.mark.parametrize("batch,h_kv,k", [(40, 4, 3), (25, 8, 7), (80, 2, 1)])
def test_listed_decode_of_many_units(batch, h_kv, k):
    # at least one unit to an SM: a CTA each, some with fewer entries than
    # warps; sequences from empty to longer than the list
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 200, batch)]
    rec, table = case(rng, lens, h_kv)
    q = queries(rng, batch, 4 * h_kv)
    idx = selection(rng, lens, h_kv, max(k, 2))[:, :, :k].copy()
    o, lse, st = run_decode(q, rec, table, lens, idx, k)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, idx))


def test_unordered_lists_with_gaps():
    rng = np.random.default_rng(7)
    lens, h_kv, k = [500, 100], 2, 20
    rec, table = case(rng, lens, h_kv)
    idx = selection(rng, lens, h_kv, k)
    for row in idx.reshape(-1, k):
        rng.shuffle(row)
    idx[1, 1] = -1                                # a list of nothing
    q = queries(rng, 2, 8)
    o, lse, st = run_decode(q, rec, table, lens, idx, k)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, idx))
    assert torch.isneginf(lse[1, 4:]).all()


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 30.0, 1e6])
def test_extreme_queries(q_scale):
    # from weights all alike to one token taking all of it
    rng = np.random.default_rng(8)
    lens = [400, 35]
    rec, table = case(rng, lens, 2)
    q = queries(rng, 2, 8, q_scale)
    o, lse, st = run_decode(q, rec, table, lens)
    assert st == 0 and torch.isfinite(o.float()).all()
    qn = q.double().numpy()
    want = Q.decode(qn, rec, table, lens)
    if q_scale <= 1e-3:
        check(o, lse, qn, rec, want)
    else:
        # scores too large for dx: only the sums' consistency is left,
        # o within the convex hull of the values, lse to fp32
        assert (np.abs(o.double().cpu().numpy()) <=
                want[2].max() * 2 + 1).all()
        np.testing.assert_allclose(lse.double().cpu().numpy(), want[1],
                                   rtol=2.0 ** -16)


def test_rows_of_very_different_scales():
    # value scales over 2^+-12 and key scales over 2^+-3: weights and value
    # exponents share one reference
    rng = np.random.default_rng(9)
    lens = [260, 700, 16]
    rec, table = case(rng, lens, 2)
    e = rec[..., 4096:].astype(np.int64)
    e[..., :16] = 127 - 9 + rng.integers(-3, 4, e[..., :16].shape)
    e[..., 16:] = 127 + rng.integers(-12, 13, e[..., 16:].shape)
    rec[..., 4096:] = e.astype(np.uint8)
    q = queries(rng, 3, 8)
    o, lse, st = run_decode(q, rec, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens))


def test_a_rising_sequence_of_scores():
    # each token scores above all before it: the reference is raised all
    # along the list
    rng = np.random.default_rng(10)
    L = 640
    rec, table = case(rng, [L], 1)
    for t in range(L):
        r = rec[table[0, t // 16], 0]
        codes, _ = Q.quantise_rows(np.full((1, 128), 448.0))
        r[Q._PLACE[t % 16]] = codes[0]
        r[4096 + t % 16] = 127 - 9
    q = torch.ones(1, 4, 128, dtype=torch.bfloat16)
    # 128 * 0.875 * 2^e / sqrt(128) = 9.9 * 2^e: rises by powers of two
    for t in range(L):
        rec[table[0, t // 16], 0, 4096 + t % 16] = 127 - 9 - 20 + t // 30
    o, lse, st = run_decode(q, rec, table, [L])
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, [L]))


def test_not_a_number_is_carried_to_its_rows_only():
    rng = np.random.default_rng(11)
    lens = [100, 100]
    rec, table = case(rng, lens, 2)
    rec[table[0, 2], 1, Q._PLACE[3]] = 0x7F        # keys of one head
    rec[table[1, 2], 0, 2048 + Q._PLACE[3, 17]] = 0x7F   # one value
    q = queries(rng, 2, 8)
    o, lse, st = run_decode(q, rec, table, lens)
    assert st == 0
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4].float()).all()
    nan = torch.isnan(o[1, :4])
    assert nan[:, 17].all() and int(nan.sum()) == 4
    assert torch.isfinite(o[1, 4:].float()).all()
    assert torch.isfinite(lse[1]).all()


def test_decode_reports_bad_data():
    rng = np.random.default_rng(12)
    lens, h_kv, k = [100, 90], 2, 4
    rec, table = case(rng, lens, h_kv)
    q = queries(rng, 2, 8)
    qn = q.double().numpy()
    idx = selection(rng, lens, h_kv, k)
    bad = idx.copy()
    bad[0, 1, 2] = 7                               # the page past the end
    o, lse, st = run_decode(q, rec, table, lens, bad, k)
    assert st == B.DEV_BAD_INDEX
    bad[0, 1, 2] = -1
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, bad))
    t2 = table.copy()
    t2[1, 0] = rec.shape[0]
    o, lse, st = run_decode(q, rec, t2, lens, idx, k)
    assert st == B.DEV_BAD_PAGE_ID
    less = idx.copy()
    less[1][less[1] == 0] = -1
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, less))
    for n, shown in ((-5, 0), (16 * table.shape[1] + 1, 16 * table.shape[1])):
        o, lse, st = run_decode(q, rec, table, [lens[0], n])
        assert st == B.DEV_BAD_SEQ_LEN
    o, lse, st = run_decode(q, rec, table, [lens[0], -5])
    check(o, lse, qn, rec, Q.decode(qn, rec, table, [lens[0], 0]))


def run_prefix(q, rec, prefix, table, lens, stream=None, ws=None):
    batch, h_q, _ = q.shape
    o = torch.full((batch, h_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((batch, h_q), 7.0, device=DEV)
    if ws is None:
        ws = B.new_prefix_workspace(batch, h_q, rec.shape[1], table.shape[1],
                                    len(prefix), DEV)
    B.locks_prefix_decode(q.to(DEV), torch.from_numpy(rec).to(DEV),
                          i32(prefix), i32(table), i32(lens), o, lse, ws,
                          stream=stream)
    torch.cuda.synchronize()
    return o, lse, B.locks_read_status(ws)


def prefix_case(rng, np_, lens, h_kv, spread=2):
    """Tables whose first np_ entries are rubbish, the prefix elsewhere."""
    rec, table = case(rng, lens, h_kv, spread)
    extra = records(rng, max(np_, 1), h_kv, spread)
    prefix = rec.shape[0] + rng.permutation(max(np_, 1))[:np_]
    table = table.copy()
    table[:, :np_] = -77
    return np.concatenate([rec, extra]), prefix.astype(np.int32), table


@pytest.mark.parametrize("G", [1, 3, 4, 8, 16])
@pytest.mark.parametrize("np_,lens,h_kv", [
    (1, [16], 1), (1, [17, 16, 40], 2), (3, [48, 49, 300, 64], 2),
    (8, [128, 200], 1), (9, [145, 144, 160], 2), (21, [336, 337, 400], 1),
    (40, [641, 700, 655, 640, 800], 2), (0, [5, 0, 40], 2),
    (6, [200, 95, 0, 1, 96, 50], 2)])
def test_prefix(G, np_, lens, h_kv):
    rng = np.random.default_rng(G * 100 + np_)
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    q = queries(rng, len(lens), G * h_kv)
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, prefix=prefix))


# enough pages times units that the prefix is taken once for all
SHARED = [(256, 1, 8, 12), (240, 2, 8, 13), (31, 16, 4, 200), (6, 5, 8, 515),
          (2, 8, 8, 1543), (64, 4, 1, 400), (100, 3, 3, 83)]
# .. and that a CTA takes two tiles of rows; an odd number of them, a last one
# with few rows
WIDE = [(67, 16, 2, 905), (129, 16, 4, 300)]


@pytest.mark.parametrize("batch,G,h_kv,np_", [
    (33, 4, 2, 70), (70, 8, 1, 20), (9, 16, 3, 130), (1, 4, 8, 3100),
    (5, 16, 1, 7001)] + SHARED + WIDE)
def test_prefix_of_many_rows(batch, G, h_kv, np_):
    # several tiles of query rows, several splits of the prefix, partial tiles
    # of both; some sequences shorter than the prefix, one empty
    rng = np.random.default_rng(batch)
    lens = [16 * np_ + int(x) for x in rng.integers(0, 60, batch)]
    lens[batch // 2] = 16 * np_ - 3
    lens[0] = 0 if batch > 20 else 16 * np_
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    q = queries(rng, batch, G * h_kv)
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, prefix=prefix))


def prefix_extremes(kind, batch, G, h_kv, np_):
    rng = np.random.default_rng(len(kind))
    lens = [16 * np_ + int(x) for x in rng.integers(0, 20, batch)]
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    q = queries(rng, batch, G * h_kv,
                {"large q": 1e15, "small q": 1e-25}.get(kind, 1.0))
    if kind == "large q":          # .. against keys that undo it
        rec[prefix, :, 4096:4112] = 127 - 32
        rec[table[:, np_:][table[:, np_:] >= 0], :, 4096:4112] = 127 - 32
        q = (q.float() * 2.0 ** -26).to(torch.bfloat16)
    if kind == "strong":           # for one row of queries, in the prefix
        r = rec[prefix[111]]
        for h in range(h_kv):
            codes, e = Q.quantise_rows(
                4 * q[7, G * h:G * h + 1].double().numpy())
            r[h, Q._PLACE[5]] = codes[0]
            r[h, 4096 + 5] = e[0] + 127
    if kind == "scales":           # rows of very different scales in a page
        e = rec[prefix][..., 4096:].astype(np.int64)
        e[..., :16] = 127 - 9 + rng.integers(-3, 4, e[..., :16].shape)
        e[..., 16:] = 127 + rng.integers(-7, 8, e[..., 16:].shape)
        tmp = rec[prefix]
        tmp[..., 4096:] = e.astype(np.uint8)
        rec[prefix] = tmp
    if kind == "rising":           # scores rise along the prefix
        codes, _ = Q.quantise_rows(np.full((1, 128), 448.0))
        for i, p in enumerate(prefix):
            for s in range(16):
                rec[p, :, Q._PLACE[s]] = codes[0][:, None]
                rec[p, :, 4096 + s] = 127 - 29 + 20 * i // np_
        q = torch.ones_like(q)
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    qn = q.double().numpy()
    # weights are off by at most 2^-25 where the largest is 2^8 or more, times
    # codes up to 448 and the largest value scale (2^-7), in each of the tokens
    below = max(lens) * 2.0 ** -33 * 448 * 2.0 ** -7 if kind == "strong" else 0
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, prefix=prefix),
          below)


EXTREMES = ["strong", "scales", "rising", "large q", "small q"]


@pytest.mark.parametrize("kind", EXTREMES)
def test_shared_prefix_extremes(kind):
    prefix_extremes(kind, 31, 4, 4, 200)


@pytest.mark.parametrize("kind", EXTREMES)
def test_shared_prefix_extremes_of_many_rows(kind):
    # enough rows and pages for two row tiles to a CTA, the last one alone
    prefix_extremes(kind, 67, 16, 2, 900)


@pytest.mark.parametrize("batch,G,h_kv,np_", [(6, 5, 8, 515),
                                              (67, 16, 2, 905)])
def test_shared_prefix_repeats_itself(batch, G, h_kv, np_):
    # buffers that are copied to while others are read: the same bits each time
    rng = np.random.default_rng(batch)
    lens = [16 * np_ + int(x) for x in rng.integers(0, 60, batch)]
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    q = queries(rng, batch, G * h_kv).to(DEV)
    rec = torch.from_numpy(rec).to(DEV)
    ws = B.new_prefix_workspace(batch, G * h_kv, h_kv, table.shape[1], np_,
                                DEV)
    prefix, table, lens = i32(prefix), i32(table), i32(lens)
    differ = torch.zeros((), dtype=torch.int32, device=DEV)
    for i in range(200):
        o = torch.zeros_like(q)
        lse = torch.zeros(q.shape[:2], device=DEV)
        B.locks_prefix_decode(q, rec, prefix, table, lens, o, lse, ws)
        if i == 0:
            first = o.clone(), lse.clone()
        differ += (o != first[0]).any() | (lse != first[1]).any()
    assert int(differ) == 0
    assert B.locks_read_status(ws) == 0


def test_shared_prefix_reports_bad_pages():
    batch, G, h_kv, np_ = 31, 4, 4, 203
    rng = np.random.default_rng(22)
    lens = [16 * np_ + int(x) for x in rng.integers(0, 20, batch)]
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    q = queries(rng, batch, G * h_kv)
    qn = q.double().numpy()
    bad = prefix.copy()
    gone = [0, 9, 17] + list(range(64, 72)) + [202]
    bad[gone] = [-1, rec.shape[0], 2 ** 31 - 1] + [-5] * 8 + [rec.shape[0]]
    # the poison of a page left out must not reach anything
    rec[prefix[gone]] = 0x7F
    o, lse, st = run_prefix(q, rec, bad, table, lens)
    assert st == B.DEV_BAD_PAGE_ID
    idx = np.tile(np.arange(np_ + 2, dtype=np.int32), (batch, h_kv, 1))
    idx[:, :, gone] = -1
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, idx, prefix))


def test_shared_prefix_does_not_mix_rows():
    # NaN queries of one sequence, and NaN keys of one head, stay there
    batch, G, h_kv, np_ = 31, 4, 4, 200
    rng = np.random.default_rng(23)
    lens = [16 * np_ + 5] * batch
    rec, prefix, table = prefix_case(rng, np_, lens, h_kv)
    rec[prefix[70], 2, Q._PLACE[3]] = 0x7F
    q = queries(rng, batch, G * h_kv)
    q[9, 4:8] = float("nan")
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    nan = torch.isnan(lse).cpu()
    want = torch.zeros_like(nan)
    want[:, 8:12] = True
    want[9, 4:8] = True
    assert torch.equal(nan, want)
    assert torch.equal(torch.isnan(o).any(-1).cpu(), want)


def test_prefix_with_one_strong_token():
    # one token far above the rest, in the prefix or in a sequence's own part
    rng = np.random.default_rng(14)
    np_, lens = 30, [500, 481, 560]
    rec, prefix, table = prefix_case(rng, np_, lens, 2)
    q = queries(rng, 3, 8)
    for pg, s in ((prefix[11], 5), (table[2, 31], 9)):
        r = rec[pg]
        for h in range(2):
            codes, e = Q.quantise_rows(4 * q[2, 4 * h:4 * h + 1].double()
                                       .numpy())
            r[h, Q._PLACE[s]] = codes[0]
            r[h, 4096 + s] = e[0] + 127
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, prefix=prefix))


def test_prefix_rows_of_very_different_scales():
    rng = np.random.default_rng(15)
    np_, lens = 20, [340, 330]
    rec, prefix, table = prefix_case(rng, np_, lens, 2)
    e = rec[..., 4096:].astype(np.int64)
    live = e < 255
    e[..., :16] = np.where(live[..., :16], 127 - 9 +
                           rng.integers(-3, 4, e[..., :16].shape), 255)
    e[..., 16:] = np.where(live[..., 16:], 127 +
                           rng.integers(-6, 7, e[..., 16:].shape), 255)
    rec[..., 4096:] = e.astype(np.uint8)
    q = queries(rng, 2, 8)
    o, lse, st = run_prefix(q, rec, prefix, table, lens)
    assert st == 0
    qn = q.double().numpy()
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, prefix=prefix))


def test_prefix_reports_bad_data():
    rng = np.random.default_rng(16)
    np_, lens = 12, [200, 260, 230]
    rec, prefix, table = prefix_case(rng, np_, lens, 2)
    q = queries(rng, 3, 8)
    qn = q.double().numpy()
    bad = prefix.copy()
    bad[[3, 9]] = [-1, rec.shape[0]]
    o, lse, st = run_prefix(q, rec, bad, table, lens)
    assert st == B.DEV_BAD_PAGE_ID
    # the pages are left out
    idx = np.tile(np.arange(17, dtype=np.int32), (3, 2, 1))
    idx[:, :, [3, 9]] = -1
    check(o, lse, qn, rec, Q.decode(qn, rec, table, lens, idx, prefix))
    o, lse, st = run_prefix(q, rec, prefix, table, [200, -1, 10 ** 6])
    assert st == B.DEV_BAD_SEQ_LEN


# ---------------------------------------------------------------------------
# streams, graphs, the whole path
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("np_,batch", [(10, 2), (200, 62)])
def test_other_stream_and_repeated_calls(np_, batch):
    rng = np.random.default_rng(17)
    lens = [16 * np_ + int(x) for x in rng.integers(0, 150, batch)]
    rec, prefix, table = prefix_case(rng, np_, lens, 2)
    q = queries(rng, batch, 8)
    o, lse, _ = run_prefix(q, rec, prefix, table, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = B.new_prefix_workspace(batch, 8, 2, table.shape[1], np_, DEV)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):                 # a used workspace, another stream
        o2, lse2, st = run_prefix(q, rec, prefix, table, lens, s, ws)
        assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("np_,batch", [(9, 3), (200, 62)])
def test_step_as_a_graph(np_, batch):
    # write one token per sequence, then attend, replayed with new inputs
    rng = np.random.default_rng(18)
    h_kv, G = 2, 4
    lens = 16 * np_ + rng.integers(0, 60, batch)
    rec, prefix, table = prefix_case(rng, np_, [int(x) + 3 for x in lens],
                                     h_kv)
    cache = torch.from_numpy(rec).to(DEV)
    t, p, L = i32(table), i32(prefix), i32(lens)
    seq = torch.arange(batch, dtype=torch.int32, device=DEV)
    k = torch.zeros(batch, h_kv, 128, dtype=torch.bfloat16, device=DEV)
    v, q = torch.zeros_like(k), torch.zeros(batch, h_kv * G, 128,
                                            dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(batch, h_kv * G, device=DEV)
    ws = B.new_prefix_workspace(batch, h_kv * G, h_kv, table.shape[1], np_,
                                DEV)

    def step():
        B.locks_quantise_kv(k, v, seq, L, t, cache, status=ws[:4].view(
            torch.int32))
        L.add_(1)
        B.locks_prefix_decode(q, cache, p, t, L, o, lse, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        L.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = rec.copy()
    for i in range(3):
        kn, vn = (torch.from_numpy(rng.standard_normal((batch, h_kv, 128)))
                  .to(torch.bfloat16) for _ in range(2))
        qn = queries(rng, batch, h_kv * G)
        k.copy_(kn)
        v.copy_(vn)
        q.copy_(qn)
        graph.replay()
        Q.write(want, kn.double().numpy(), vn.double().numpy(), range(batch),
                lens + i, table)
        torch.cuda.synchronize()
        qd = qn.double().numpy()
        check(o, lse, qd, want, Q.decode(qd, want, table, lens + i + 1,
                                         prefix=prefix))
    assert B.locks_read_status(ws) == 0


def test_summaries_from_pages_read_back():
    # the keys read back are a bf16 cache: summaries built from them equal
    # those built from a bf16 cache of the same numbers
    rng = np.random.default_rng(19)
    h_kv, L = 2, 70
    table = np.array([[4, 1, 3, 0, 2]], np.int32)
    k = torch.from_numpy(rng.standard_normal((L, h_kv, 128))) \
        .to(DEV, torch.bfloat16)
    cache = B.new_quantised_cache(5, h_kv, DEV)
    B.locks_quantise_kv(k, k, i32([0] * L), i32(range(L)), i32(table), cache)
    pages = i32(range(4))
    zero = i32([0] * 4)
    keys = torch.empty(4, h_kv, 16, 128, dtype=torch.bfloat16, device=DEV)
    B.locks_dequantise_kv(cache, i32(table), zero, pages, keys, None)
    store = B.new_summary_store(1, h_kv, 4, DEV)
    B.locks_build_summaries(keys, pages.view(1, 4), zero, pages, store)
    ostore, _ = O.build_summaries(keys.float().cpu().numpy(),
                                  np.arange(4)[None], [0] * 4, range(4), 1, 4)
    a = O.decode_records(store.cpu().numpy().reshape(-1, 832))
    b = O.decode_records(np.asarray(ostore).reshape(-1, 832))
    for part in ("mu8", "smu"):
        np.testing.assert_array_equal(a[part], b[part])


def test_example_runs_them_together():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "quantised_cache.py")
    spec = importlib.util.spec_from_file_location("quantised_cache", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # some pages selected, then all: where the lists hold every page the two
    # attentions are the same sums, each rounded to bf16 once (2^-8 of the
    # value apiece) after weights of 2^-11
    s, mass = example.main(batch=4, h_q=8, h_kv=2, doc_pages=40, k=12,
                           steps=20, show=lambda _: None)
    assert s.bad() == 0 and 0.1 < mass < 1.0
    s, mass = example.main(batch=4, h_q=8, h_kv=2, doc_pages=40, k=50,
                           steps=17, show=lambda _: None)
    assert s.bad() == 0
    (o, lse), (o2, lse2) = s.outs
    K, V = Q.read(s.cache.cpu().numpy())
    tol = 2.0 ** -7 * o.abs().max() + 2.0 ** -10 * float(np.abs(V).max())
    assert (o.float() - o2.float()).abs().max() <= tol
    assert (lse - lse2).abs().max() <= 1e-4
