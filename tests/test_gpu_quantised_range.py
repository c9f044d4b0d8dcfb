"""GPU tests of the quantised KV cache at the limits of what its calls take:
batches, scales, queries."""
import math

import numpy as np
import pytest
import torch

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


def records(rng, P, h_kv, spread=2, centre=-9):
    """Random records: any finite codes, scales around 2^centre."""
    rec = rng.integers(0, 256, (P, h_kv, Q.RECORD)).astype(np.uint8)
    codes = rec[..., :4096]
    codes[(codes & 0x7F) == 0x7F] = 0x10
    rec[..., 4096:] = 127 + centre + rng.integers(-spread, spread + 1,
                                                  rec[..., 4096:].shape)
    return rec


# ---------------------------------------------------------------------------
# batches
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("batch", [40959, 40960, 41088])
@pytest.mark.parametrize("np_", [0, 1])
def test_largest_batches(batch, np_):
    # the form that keeps a prefix sum of all sequences on chip (tables too
    # long for a unit to a CTA), alone and beside the shared prefix's kernel;
    # five kinds of sequences, all of a kind alike
    rng = np.random.default_rng(np_)
    lens, max_pages = [16 * np_ + n for n in (0, 1, 16, 17, 40)], 66
    rec = records(rng, 20, 1)
    tables = rng.integers(0, 20, (5, max_pages)).astype(np.int32)
    tables[:, :np_] = 3
    q = torch.from_numpy(rng.standard_normal((5, 2, 128))).to(torch.bfloat16)
    kind = torch.arange(batch, device=DEV) % 5
    qd, table, seq_lens = q.to(DEV)[kind], i32(tables)[kind], i32(lens)[kind]
    cache = torch.from_numpy(rec).to(DEV)
    o = torch.full((batch, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((batch, 2), 7.0, device=DEV)
    ws = B.new_prefix_workspace(batch, 2, 1, max_pages, np_, DEV)
    if np_:
        B.locks_prefix_decode(qd, cache, i32([3]), table, seq_lens, o, lse, ws)
    else:
        B.locks_quantised_decode(qd, cache, table, seq_lens, None, max_pages,
                                 o, lse, ws)
    assert B.locks_read_status(ws) == 0
    want, wlse, mass = Q.decode(q.double().numpy(), rec, tables, lens)
    # weights of 2^-11, exponentials and sums of 2^-13, o rounded to bf16
    # once; scores of 128 products of 2^-24 each
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -13) * mass + 1e-30
    for k in range(5):
        got = o[k::5].double().cpu().numpy()
        assert (np.abs(got - want[k]) <= tol[k]).all()
        got = lse[k::5].double().cpu().numpy()
        if np.isneginf(wlse[k]).all():
            assert np.isneginf(got).all()
        else:
            assert (np.abs(got - wlse[k]) <= 1e-4).all()


# ---------------------------------------------------------------------------
# order
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("batch,np_", [(62, 200), (3, 9)])
def test_steps_back_to_back_see_the_latest_inputs(batch, np_):
    # queries, lengths, tables and rows change right before every call, with
    # nothing between the kernels; the kernel of the sequences' own pages
    # starts before the prefix's has ended and reads them
    rng = np.random.default_rng(batch)
    h_kv, G, steps, max_pages = 2, 4, 24, np_ + 5
    P = np_ + batch * 5
    rec = torch.from_numpy(records(rng, P, h_kv)).to(DEV)
    prefix = i32(rng.permutation(np_))
    tables = i32(np.stack([np.concatenate(
        [np.full((batch, np_), -7),
         np_ + rng.permutation(batch * 5).reshape(batch, 5)], 1)
        for _ in range(steps)]))
    lens = i32(16 * np_ + rng.integers(0, 70, (steps, batch)))
    q = torch.from_numpy(rng.standard_normal((steps, batch, h_kv * G, 128))) \
        .to(DEV, torch.bfloat16)
    kv = torch.from_numpy(rng.standard_normal((steps, batch, h_kv, 128))) \
        .to(DEV, torch.bfloat16)
    seq = torch.arange(batch, dtype=torch.int32, device=DEV)

    def run(wait):
        cache, table, L = rec.clone(), tables[0].clone(), lens[0].clone()
        row, qi = kv[0].clone(), q[0].clone()
        ws = B.new_prefix_workspace(batch, h_kv * G, h_kv, max_pages, np_, DEV)
        outs = [(torch.empty_like(qi), torch.empty(batch, h_kv * G,
                                                   device=DEV))
                for _ in range(steps)]
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(outs):
            for to, new in ((table, tables[i]), (row, kv[i]), (qi, q[i]),
                            (L, lens[i])):
                to.copy_(new)
            B.locks_quantise_kv(row, row, seq, L, table, cache)
            if wait:
                torch.cuda.synchronize()
            L.add_(1)
            if wait:
                torch.cuda.synchronize()
            B.locks_prefix_decode(qi, cache, prefix, table, L, o, lse, ws)
            if wait:
                torch.cuda.synchronize()
        assert B.locks_read_status(ws) == 0
        return outs

    want = run(True)
    for _ in range(5):
        for (o, lse), (wo, wl) in zip(run(False), want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


# ---------------------------------------------------------------------------
# values of very different scales
# ---------------------------------------------------------------------------
# Tolerances, per output element, from the formats:
#   * o rounded to bf16 once: half a step, 2^-8 of it
#   * every weight rounded to 11 bits or more, whatever its size, exponentials
#     and fp32 sums: 2^-11 + 2^-13 of each term p |v|
#   * rows whose scale is within 2^8 of the largest keep fp16 weights, off by
#     2^-25 at most where the largest term's is 2^8 or more: 2^-33 of the
#     largest weight times the largest scale, 2^-25 of it times the row's own
#   * scores off by dx each: a weight by expm1(2 max dx) of it, the largest
#     weight by as much of all the others'
#   * dx: 128 products and sums, 2^-24 each; fp32 exponents of numbers up to
#     |x| + 64, twice; the query as the call takes it (`query`: an element's
#     error, as a share of the row's largest, or of each element by itself)
#   * lse: max dx, fp32 rounding
# Outputs in dims where the far larger rows hold zeros are sums of the others
# alone, so these hold element by element, not against the row's largest.
def bounds(q, K, V, query):
    G = q.shape[0]
    if K.shape[0] == 0:
        return (np.zeros((G, 128)), np.full(G, -np.inf), np.zeros((G, 128)),
                np.zeros(G))
    x = q @ K.T / math.sqrt(128)
    off = query(q) if callable(query) else np.broadcast_to(
        query * np.abs(q).max(1, keepdims=True), q.shape)
    dx = (2.0 ** -17 * np.abs(q) + off) @ np.abs(K).T / math.sqrt(128)
    dx = (dx + 2.0 ** -22 * (np.abs(x) + 64)).max(1)
    top = x.max(1, keepdims=True)
    w = np.exp(x - top)
    total = w.sum(1, keepdims=True)
    p = w / total
    o, lse = p @ V, (top + np.log(total))[:, 0]
    absv = np.abs(V)
    best = p.argmax(1)
    rest = p.copy()
    rest[np.arange(G), best] = 0.0
    move = np.expm1(np.minimum(2 * dx, 50.0))[:, None]
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * (p @ absv) + \
        2.0 ** -25 * p.max(1)[:, None] * absv.sum(0) + \
        move * (rest @ absv + rest.sum(1)[:, None] * absv[best]) + 1e-36
    return o, lse, tol, dx + 2.0 ** -20 * np.abs(lse) + 2.0 ** -20


def expect(got, q, rec, tables, lens, idx=None, prefix=None, query=2.0 ** -32):
    """Every output of a decode against the definition in 64 bits."""
    got_o, got_lse = (t.double().cpu().numpy() for t in got)
    h_kv = rec.shape[1]
    G = q.shape[1] // h_kv
    np_ = 0 if prefix is None else len(prefix)
    for h in range(h_kv):
        if np_:
            K0, V0 = Q.read(rec[prefix, h])
            K0, V0 = K0.reshape(-1, 128), V0.reshape(-1, 128)
        for b, n in enumerate(lens):
            n = int(n)
            pages = range(np_, -(-n // 16)) if idx is None else idx[b, h]
            K, V = Q.tokens(rec, tables[b], h, pages, n)
            if np_:
                K = np.concatenate([K0[:n], K])
                V = np.concatenate([V0[:n], V])
            sl = slice(h * G, (h + 1) * G)
            o, lse, tol, ltol = bounds(q[b, sl], K, V, query)
            off = np.abs(got_o[b, sl] - o)
            bad = np.argwhere(~(off <= tol))
            assert len(bad) == 0, (b, h, len(bad), bad[:4],
                                   (off / tol).max())
            if K.shape[0] == 0:
                assert np.isneginf(got_lse[b, sl]).all()
            else:
                assert (np.abs(got_lse[b, sl] - lse) <= ltol).all(), (b, h)


def layout(rng, lens, h_kv, centre, room=2, np_=0):
    """Records with value scales around 2^centre, tables; NaN and absurd
    scales past each sequence's end."""
    batch = len(lens)
    max_pages = max(1, -(-max(lens) // 16)) + room
    P = batch * (max_pages - np_) + np_ + 3
    perm = rng.permutation(P).astype(np.int32)
    prefix = perm[:np_]
    tables = np.full((batch, max_pages), -77, np.int32)
    tables[:, np_:] = perm[np_:np_ + batch * (max_pages - np_)].reshape(
        batch, -1)
    rec = records(rng, P, h_kv)
    rec[..., 4112:] = 127 + centre + rng.integers(-2, 3, rec[..., 4112:].shape)
    for b, n in enumerate(lens):
        if n % 16 and n // 16 >= np_:
            r = rec[tables[b, n // 16]]
            for s in range(n % 16, 16):
                r[:, Q._PLACE[s]] = r[:, 2048 + Q._PLACE[s]] = 0x7F
                r[:, [4096 + s, 4112 + s]] = 255
    return rec, tables, prefix


def plant(rec, page, slot, exponent, dims=(17,), q=None):
    """Gives a row the value 448 * 2^exponent in `dims` and zero elsewhere,
    and with `q` [h_kv][128] a key that scores high with these."""
    for h in range(rec.shape[1]):
        r = rec[page, h]
        r[2048 + Q._PLACE[slot]] = 0
        r[2048 + Q._PLACE[slot, list(dims)]] = 0x7E
        r[4112 + slot] = 127 + exponent
        if q is not None:
            codes, e = Q.quantise_rows(q[h][None])
            r[Q._PLACE[slot]] = codes[0]
            r[4096 + slot] = e[0] + 127


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16)


def run_lists(q, rec, tables, lens, idx=None):
    batch, h_q, _ = q.shape
    max_pages = tables.shape[1]
    k = max_pages if idx is None else idx.shape[2]
    o = torch.full((batch, h_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((batch, h_q), 7.0, device=DEV)
    ws = B.new_workspace(batch, h_q, rec.shape[1], max_pages, k, DEV)
    B.locks_quantised_decode(q.to(DEV), torch.from_numpy(rec).to(DEV),
                             i32(tables), i32(lens),
                             None if idx is None else i32(idx), k, o, lse, ws)
    assert B.locks_read_status(ws) == 0
    return o, lse


def lists(rng, lens, h_kv, k):
    idx = np.full((len(lens), h_kv, k), -1, np.int32)
    for b, n in enumerate(lens):
        n = -(-n // 16)
        for h in range(h_kv):
            some = rng.permutation(n)[:k]
            some[:2] = [0, n - 1]
            some = np.unique(some)
            idx[b, h, :len(some)] = some
    return idx


FORMS = [([640, 500, 17], 2, 0, 0), ([900, 33], 2, 600, 0),
         ([2000, 1500], 2, 2, 40)]   # lens, h_kv, room, k


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("lens,h_kv,room,k", FORMS)
@pytest.mark.parametrize("centre,high", [(-9, 15), (-9, 31), (-30, 31)])
@pytest.mark.parametrize("strong", [False, True])
def test_one_value_far_above_the_rest(G, lens, h_kv, room, k, centre, high,
                                      strong):
    # scales 24, 40 and 61 apart (a CTA to a unit, runs over all lists,
    # clusters): the high row first, in the middle and last, among ordinary
    # weights or with most of the weight of one query head
    rng = np.random.default_rng(G + high)
    rec, tables, _ = layout(rng, lens, h_kv, centre, room)
    q = normal(rng, len(lens), G * h_kv, 128)
    qn = q.double().numpy()
    for b, n in enumerate(lens):
        t = (0, n // 2, n - 1)[b]
        plant(rec, tables[b, t // 16], t % 16, high, q=0.7 * qn[b, ::G]
              if strong else None)
    idx = lists(rng, lens, h_kv, k) if k else None
    expect(run_lists(q, rec, tables, lens, idx), qn, rec, tables, lens, idx)


@pytest.mark.parametrize("G", [1, 8, 12])
@pytest.mark.parametrize("room", [0, 700])
def test_values_of_the_whole_scale_range(G, room):
    # every row its own scale in -32 .. 31
    rng = np.random.default_rng(G)
    lens = [500, 31, 700]
    rec, tables, _ = layout(rng, lens, 2, 0, room)
    live = rec[..., 4112:] < 255
    rec[..., 4112:] = np.where(
        live, 127 + rng.integers(-32, 32, live.shape), 255)
    # few codes that are not zero, so that every dim has rows of its own
    codes = rec[..., 2048:4096]
    codes[rng.random(codes.shape) < 0.99] = 0
    q = normal(rng, 3, G * 2, 128)
    qn = q.double().numpy()
    # rubbish past the ends again
    for b, n in enumerate(lens):
        for s in range(n % 16, 16):
            rec[tables[b, n // 16], :, 2048 + Q._PLACE[s]] = 0x7F
    expect(run_lists(q, rec, tables, lens), qn, rec, tables, lens)


@pytest.mark.parametrize("value", [math.inf, -math.inf, 1e9, 1e8, 1e6])
def test_attention_over_rows_with_one_huge_number(value):
    # written by the framework itself: infinities are kept as +-448 * 2^31
    rng = np.random.default_rng(5)
    n, h_kv, G = 512, 2, 4
    k, v = normal(rng, n, h_kv, 128), normal(rng, n, h_kv, 128)
    v[100, :, 5] = value
    table = i32(np.arange(32)[None])
    cache = B.new_quantised_cache(32, h_kv, DEV)
    B.locks_quantise_kv(k.to(DEV), v.to(DEV), i32([0] * n), i32(range(n)),
                        table, cache)
    rec, tables = cache.cpu().numpy(), table.cpu().numpy()
    q = normal(rng, 1, G * h_kv, 128)
    expect(run_lists(q, rec, tables, [n]), q.double().numpy(), rec, tables,
           [n])


def run_shared(q, rec, tables, lens, prefix, shared=True):
    """locks_prefix_decode; `shared`: the prefix's own kernel has to be among
    the three that run (its form is chosen by sizes)."""
    batch, h_q, _ = q.shape
    o = torch.full((batch, h_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((batch, h_q), 7.0, device=DEV)
    ws = B.new_prefix_workspace(batch, h_q, rec.shape[1], tables.shape[1],
                                len(prefix), DEV)
    args = (q.to(DEV), torch.from_numpy(rec).to(DEV), i32(prefix),
            i32(tables), i32(lens), o, lse, ws)
    before = B.lib().locks_kernel_launches()
    B.locks_prefix_decode(*args)
    assert (B.lib().locks_kernel_launches() - before == 3) == shared
    assert B.locks_read_status(ws) == 0
    return o, lse


# batch, G, h_kv, pages: ranges of one tile (128 tokens) with one tile of 128
# query rows to a CTA; ranges of several; two tiles of query rows
SHARED = [(31, 4, 4, 200), (6, 5, 8, 515), (67, 16, 2, 905)]


def shared_case(rng, batch, G, h_kv, np_, centre):
    lens = [16 * np_ + int(n) for n in rng.integers(0, 40, batch)]
    lens[1] = 16 * np_ - 5             # shorter than the prefix
    lens[3] = 16 * np_ + 20
    rec, tables, prefix = layout(rng, lens, h_kv, centre, np_=np_)
    q = normal(rng, batch, G * h_kv, 128)
    return rec, tables, prefix, lens, q, q.double().numpy()


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
@pytest.mark.parametrize("centre,high", [(-9, 15), (-9, 31), (-30, 31)])
@pytest.mark.parametrize("strong", [False, True])
def test_shared_value_far_above_the_rest(batch, G, h_kv, np_, centre, high,
                                         strong):
    # high rows in a page, a tile and a range of ordinary ones, at their
    # beginnings and ends, and one in a sequence's own part
    rng = np.random.default_rng(np_ + high)
    rec, tables, prefix, lens, q, qn = shared_case(rng, batch, G, h_kv, np_,
                                                   centre)
    key = 0.7 * qn[2, ::G] if strong else None
    for pg, slot in ((0, 0), (9, 15), (np_ // 2, 7), (np_ - 1, 15)):
        plant(rec, prefix[pg], slot, high, (17 + pg % 50,), key)
    plant(rec, tables[3, np_], 3, high, (5,))
    expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
           prefix=prefix, query=2.0 ** -18)


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
def test_shared_value_far_below_its_page(batch, G, h_kv, np_):
    # a row with nearly all of the weight of some heads, its scale 2^22 and
    # more below that of the other rows of its page, which are zero in half of
    # the dims
    rng = np.random.default_rng(np_)
    rec, tables, prefix, lens, q, qn = shared_case(rng, batch, G, h_kv, np_, 0)
    codes = rec[:, :, 2048:4096]
    for s in range(16):
        codes[:, :, Q._PLACE[s, :64]] = 0
    for pg, slot in ((3, 0), (12, 9), (np_ - 2, 15)):
        plant(rec, prefix[pg], slot, -22 - pg % 7, range(0, 128, 3),
              0.7 * qn[2, ::G])
    expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
           prefix=prefix, query=2.0 ** -18)


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
def test_shared_values_of_the_whole_scale_range(batch, G, h_kv, np_):
    rng = np.random.default_rng(np_ + 1)
    rec, tables, prefix, lens, q, qn = shared_case(rng, batch, G, h_kv, np_, 0)
    # every third page: scales in -32 .. 31; the others narrow at some level
    part = rec[prefix]
    e = part[..., 4112:].astype(np.int64)
    wide = rng.integers(-32, 32, e.shape)
    level = rng.integers(-30, 30, (np_, 1, 1)) + rng.integers(-2, 2, e.shape)
    third = (np.arange(np_) % 3 == 0)[:, None, None]
    part[..., 4112:] = 127 + np.where(third, wide, level)
    v = part[..., 2048:4096]
    v[rng.random(v.shape) < 1 - 2 / (16 * np_)] = 0   # two rows to a dim
    rec[prefix] = part
    expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
           prefix=prefix, query=2.0 ** -18)


# ---------------------------------------------------------------------------
# queries with an outlier
# ---------------------------------------------------------------------------
def shared_query_error(q):
    """hi + lo of the shared pages' query: scaled by a power of two that puts
    the row's largest in (224, 448], or [2^11, 2^12) where it is 64 times the
    mean (taken from sums of 15 additions in bf16: 15 * 2^-9 to spare), off by
    2^-14 at most below 2^-6."""
    top = np.abs(q).max(1, keepdims=True)
    unit = np.where(2 * top > 1.03 * np.abs(q).sum(1, keepdims=True),
                    2.0 ** (np.floor(np.log2(top)) - 11),
                    2.0 ** np.ceil(np.log2(top / 448)))
    return np.where(np.abs(q) < 2.0 ** -6 * unit, 2.0 ** -14 * unit, 0.0)


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
@pytest.mark.parametrize("ratio", [30, 1000, 20000])
@pytest.mark.parametrize("keys", ["alike", "apart"])
def test_shared_query_with_an_outlier_channel(batch, G, h_kv, np_, ratio,
                                              keys):
    # one element far above the rest, against keys that are small there: the
    # other elements carry the score.  With all keys alike a score's error
    # does not average out of the log-sum-exp
    rng = np.random.default_rng(ratio)
    rec, tables, prefix, lens, q, qn = shared_case(rng, batch, G, h_kv, np_,
                                                   -9)
    q[:, :, 40] *= ratio
    if keys == "apart":       # some tokens well above the others
        q *= 3
    qn = q.double().numpy()
    for h in range(h_kv):
        k = rng.standard_normal((64, 128))
        k[:, 40] /= ratio
        codes, e = Q.quantise_rows(k)
        at = np.zeros(rec.shape[0] * 16, np.int64)
        if keys == "apart":
            at = rng.integers(0, 64, at.shape)
        part = np.empty((at.size, 128), np.uint8)
        part[:] = codes[at]
        place = np.array(Q._PLACE).reshape(-1)
        rows = np.empty((rec.shape[0], 2048), np.uint8)
        rows[:, place] = part.reshape(rec.shape[0], 2048)
        rec[:, h, :2048] = rows
        rec[:, h, 4096:4112] = (127 + e[at]).reshape(-1, 16)
    expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
           prefix=prefix, query=shared_query_error)


# ---------------------------------------------------------------------------
# records never written
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("centre", [-9, 4, 25])
@pytest.mark.parametrize("G,room", [(4, 0), (4, 600), (12, 0)])
def test_zeroed_records_inside_a_length(centre, G, room):
    # a new cache is zeros, scale bytes too: keys and values of zero, which
    # have their share of the weights whatever the other rows' scales
    rng = np.random.default_rng(centre + 9)
    lens = [300, 80, 45]
    rec, tables, _ = layout(rng, lens, 2, centre, room)
    for b, pages in ((0, [1, 4, 5, 18]), (1, [0]), (2, [0, 1])):
        rec[tables[b, pages]] = 0
    q = normal(rng, 3, 2 * G, 128)
    expect(run_lists(q, rec, tables, lens), q.double().numpy(), rec, tables,
           lens)


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
@pytest.mark.parametrize("centre", [-9, 4, 25])
def test_shared_zeroed_records(batch, G, h_kv, np_, centre):
    rng = np.random.default_rng(np_)
    rec, tables, prefix, lens, q, qn = shared_case(rng, batch, G, h_kv, np_,
                                                   centre)
    rec[prefix[rng.random(np_) < 0.3]] = 0
    rec[prefix[16:40]] = 0             # whole tiles
    for b in (0, 5):                   # single rows
        for s in range(b, 16, 3):
            r = rec[prefix[7 + b]]
            r[:, Q._PLACE[s]] = r[:, 2048 + Q._PLACE[s]] = 0
            r[:, [4096 + s, 4112 + s]] = 0
    expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
           prefix=prefix, query=shared_query_error)


# ---------------------------------------------------------------------------
# scores that rise, extreme queries
# ---------------------------------------------------------------------------
def kernel_names(call):
    from torch.profiler import ProfilerActivity, profile
    for _ in range(2):       # a process's first profile may come back empty
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        names = " ".join(e.key for e in p.key_averages())
        if names:
            return names
    pytest.skip("no kernel names from the profiler")


@pytest.mark.parametrize("batch,G,h_kv,np_,tiles", [
    (2, 8, 8, 1543, 1), (67, 16, 2, 905, 2)])
def test_shared_forms(batch, G, h_kv, np_, tiles):
    # the cases below mean these forms of the kernel, chosen by sizes: one or
    # two tiles of query rows to a CTA, and at least two tiles of tokens to a
    # range (there are at most 608 CTAs with one, 304 with two)
    rng = np.random.default_rng(0)
    rec, tables, prefix, lens, q, _ = shared_case(rng, max(batch, 4), G, h_kv,
                                                  np_, -9)
    names = kernel_names(lambda: run_shared(q[:batch], rec, tables[:batch],
                                            lens[:batch], prefix))
    assert f"prefix_kernel<{tiles}>" in names
    row_tiles = -(-batch * G // 128)
    ranges = 608 // tiles / (-(-row_tiles // tiles) * h_kv)
    assert -(-np_ // 8) >= 2 * ranges


def rising_keys(rng, rec, pages, q_unit, levels):
    """Keys of page i of `pages` along q_unit [128], scoring levels[i] with
    it."""
    for i, pg in enumerate(pages):
        for s in range(16):
            x = levels[i][s] * math.sqrt(128) / (q_unit ** 2).sum()
            # the spread keeps the rounding of the codes from adding up
            k = x * q_unit * (1 + 0.1 * rng.uniform(-1, 1, (rec.shape[1], 128)))
            codes, e = Q.quantise_rows(k)
            for h in range(rec.shape[1]):
                rec[pg, h, Q._PLACE[s]] = codes[h]
                rec[pg, h, 4096 + s] = 127 + e[h]


@pytest.mark.parametrize("batch,G,h_kv,np_", [(6, 5, 8, 515), (2, 8, 8, 1543),
                                              (67, 16, 2, 905)])
@pytest.mark.parametrize("spread", [2, 14])
def test_shared_scores_that_rise(batch, G, h_kv, np_, spread):
    # along the tiles of a range and in the middle of a tile, for rows of
    # different steepness: sums and weights are rescaled again and again, in
    # tiles of either form (value scales near one another, and far apart)
    rng = np.random.default_rng(np_ + spread)
    lens = [16 * np_ + int(n) for n in rng.integers(0, 40, batch)]
    rec, tables, prefix = layout(rng, lens, h_kv, -9, np_=np_)
    if spread > 2:
        part = rec[prefix]
        part[..., 4112:] = 127 + rng.integers(-spread, spread + 1,
                                              part[..., 4112:].shape)
        rec[prefix] = part
    unit = rng.choice([-1.0, 1.0], 128)
    steep = rng.choice([0.5, 1.0, 1.5, 2.0], (batch, h_kv * G, 1))
    q = torch.from_numpy(steep * unit + 0.05 * rng.standard_normal(
        (batch, h_kv * G, 128))).to(torch.bfloat16)
    page = np.arange(np_)
    levels = 5.0 * (page // 8 % 8) + 6.0 * (page // 4 % 2) - 20
    rising_keys(rng, rec, prefix, unit,
                levels[:, None] + rng.uniform(-1, 1, (np_, 16)))
    expect(run_shared(q, rec, tables, lens, prefix), q.double().numpy(), rec,
           tables, lens, prefix=prefix, query=shared_query_error)


@pytest.mark.parametrize("lens,h_kv,room,k", FORMS)
@pytest.mark.parametrize("spread", [2, 14])
def test_scores_that_rise(lens, h_kv, room, k, spread):
    rng = np.random.default_rng(spread)
    rec, tables, _ = layout(rng, lens, h_kv, -9, room)
    live = rec[..., 4112:] < 255
    if spread > 2:
        rec[..., 4112:] = np.where(
            live, 127 + rng.integers(-spread, spread + 1, live.shape), 255)
    unit = rng.choice([-1.0, 1.0], 128)
    for b, n in enumerate(lens):
        full = tables[b, :n // 16]
        levels = 5.0 * (np.arange(len(full)) % 8) - 20
        rising_keys(rng, rec, full, unit,
                    levels[:, None] + rng.uniform(-1, 1, (len(full), 16)))
    steep = rng.choice([0.5, 1.0, 1.5, 2.0], (len(lens), h_kv * 4, 1))
    q = torch.from_numpy(steep * unit + 0.05 * rng.standard_normal(
        (len(lens), h_kv * 4, 128))).to(torch.bfloat16)
    idx = lists(rng, lens, h_kv, k) if k else None
    expect(run_lists(q, rec, tables, lens, idx), q.double().numpy(), rec,
           tables, lens, idx)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 1e3, 1e6])
@pytest.mark.parametrize("form", [0, 1, 2, "shared"])
def test_queries_of_any_size(scale, form):
    # every output against the definition: at the largest sizes one token
    # takes a row, and which one does not depend on the scores' last bits
    rng = np.random.default_rng(8)
    if form == "shared":
        rec, tables, prefix, lens, q, _ = shared_case(rng, *SHARED[1], -9)
    else:
        lens, h_kv, room, k = FORMS[form]
        rec, tables, _ = layout(rng, lens, h_kv, -9, room)
        q = normal(rng, len(lens), 4 * h_kv, 128)
    q = (scale * q.double()).to(torch.bfloat16)
    qn = q.double().numpy()
    if form == "shared":
        expect(run_shared(q, rec, tables, lens, prefix), qn, rec, tables, lens,
               prefix=prefix, query=shared_query_error)
    else:
        idx = lists(rng, lens, h_kv, k) if k else None
        expect(run_lists(q, rec, tables, lens, idx), qn, rec, tables, lens,
               idx)


# ---------------------------------------------------------------------------
# equal scores
# ---------------------------------------------------------------------------
def alike(rng, rec, places, exponent):
    """The same key, 448 * 2^exponent in dim 3, at all places (page, slot), as
    an infinity there leaves it; values of scales 2^-6 to 2^6 around 2^-9."""
    for pg, s in places:
        r = rec[pg]
        r[:, Q._PLACE[s]] = 0
        r[:, Q._PLACE[s, 3]] = 0x7E
        r[:, 4096 + s] = 127 + exponent
        r[:, 4112 + s] = 127 - 9 + rng.integers(-6, 7, rec.shape[1])


def expect_mean(got, qn, rec, places, exponent):
    """places [batch][n]: the tokens that share a row's weight equally."""
    o, lse = (t.double().cpu().numpy() for t in got)
    batch, h_q, _ = qn.shape
    h_kv = rec.shape[1]
    G = h_q // h_kv
    for b in range(batch):
        pages, slots = zip(*places[b])
        for h in range(h_kv):
            V = Q.read(rec[list(pages), h])[1][range(len(pages)), list(slots)]
            mean, mass = V.mean(0), np.abs(V).mean(0)
            tol = 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -13) * mass
            sl = slice(h * G, (h + 1) * G)
            bad = np.argwhere(~(np.abs(o[b, sl] - mean) <= tol))
            assert len(bad) == 0, (b, h, len(bad), bad[:4])
            x = qn[b, sl, 3] * 448 * 2.0 ** exponent / math.sqrt(128)
            want = x + math.log(len(pages))
            assert (np.abs(lse[b, sl] - want) <= 2.0 ** -21 * x).all()


# scores of some 80, 2e4, 2e6, 1e11
LEVELS = [1, 9, 16, 31]


@pytest.mark.parametrize("lens,h_kv,room,k", FORMS)
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("exponent", LEVELS)
def test_equal_scores_of_any_size(lens, h_kv, room, k, G, exponent):
    rng = np.random.default_rng(exponent)
    rec, tables, _ = layout(rng, lens, h_kv, -9, room)
    rec[..., 4096:4112] = np.minimum(rec[..., 4096:4112], 127 - 9)
    q = normal(rng, len(lens), G * h_kv, 128)
    q[:, :, 3] = 1 + (q[:, :, 3].abs() * 4).round().clamp(max=4) / 4
    places = []
    for b, n in enumerate(lens):
        at = [0, 3, n // 3, n // 2, n - 2, n - 1]   # pages that lists hold
        if k:
            at = [0, 3, 9, n - 1]
        places.append(sorted({(int(tables[b, t // 16]), t % 16) for t in at}))
        alike(rng, rec, places[-1], exponent)
    idx = lists(rng, lens, h_kv, k) if k else None
    expect_mean(run_lists(q, rec, tables, lens, idx), q.double().numpy(), rec,
                places, exponent)


@pytest.mark.parametrize("batch,G,h_kv,np_", SHARED)
@pytest.mark.parametrize("exponent", LEVELS)
def test_shared_equal_scores_of_any_size(batch, G, h_kv, np_, exponent):
    # in one tile, in one range, in several, and in the sequences' own pages
    rng = np.random.default_rng(exponent)
    lens = [16 * np_ + int(n) for n in rng.integers(5, 40, batch)]
    rec, tables, prefix = layout(rng, lens, h_kv, -9, np_=np_)
    q = normal(rng, batch, G * h_kv, 128)
    q[:, :, 3] = 1 + (q[:, :, 3].abs() * 4).round().clamp(max=4) / 4
    shared = [(int(prefix[t // 16]), t % 16)
              for t in (1, 14, 60, 100, 900, 8 * np_, 16 * np_ - 1)]
    alike(rng, rec, shared, exponent)
    places = []
    for b in range(batch):
        own = [(int(tables[b, np_]), b % 5)] if b % 2 else []
        alike(rng, rec, own, exponent)
        places.append(shared + own)
    expect_mean(run_shared(q, rec, tables, lens, prefix), q.double().numpy(),
                rec, places, exponent)
