"""GPU parity of rotary positions against the float64 oracle.

Tolerances.  A turned number is x cos - y sin or x sin + y cos: the angle is
off by 2^-26 turns (an fp32 number in [-1/2, 1/2]; 2 pi 2^-26 = 2^-23.3 rad),
cosine and sine by two last places more (2^-23), and two products, their sum
and the amplitude round by 2^-24 each: together below 2^-20 of |x| + |y|.  Then
one rounding to the output: bf16 2^-8 of the value, e4m3 2^-4 of it or half of
the least step, 2^-10 2^e.  Numbers that are not turned are rounded alone.
"""
import numpy as np
import pytest
import torch

from oracle import quantised_oracle as Q
from oracle import window_oracle as W
from sparse_paged_kv_locks_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def num(t):
    return t.double().cpu().numpy()


def frequencies(dim, base=10000.0):
    return [base ** (-2 * j / dim) for j in range(dim // 2)]


class Case:
    """Tokens of ragged sequences after a fused projection, with their places
    in a shuffled table."""

    def __init__(self, seed, lens, h_q, h_kv, dtype="bf16", past=3):
        rng = self.rng = np.random.default_rng(seed)
        self.n, self.h_q, self.h_kv = sum(lens), h_q, h_kv
        batch = len(lens)
        self.pages = max(1, max(-(-(x + past) // 16) for x in lens))
        x = rng.standard_normal((self.n, h_q + 2 * h_kv, 128)) * \
            2.0 ** rng.integers(-6, 6, (self.n, h_q + 2 * h_kv, 1))
        qkv = torch.from_numpy(x).to(TYPES[dtype]).to(DEV)
        self.q, self.k, self.v = qkv.split((h_q, h_kv, h_kv), 1)
        self.seq = np.repeat(np.arange(batch), lens).astype(np.int32)
        self.pos = np.concatenate([past + np.arange(x) for x in lens]).astype(
            np.int32)
        self.table = rng.permutation(batch * self.pages).astype(
            np.int32).reshape(batch, self.pages)
        self.P = batch * self.pages
        self.kc = torch.full((self.P, h_kv, 16, 128), 7.0,
                             dtype=torch.bfloat16, device=DEV)
        self.vc = torch.full_like(self.kc, 9.0)
        self.rec = torch.full((self.P, h_kv, 4128), 171, dtype=torch.uint8,
                              device=DEV)
        self.qo = torch.full((self.n, h_q, 128), 5.0, dtype=torch.bfloat16,
                             device=DEV)

    def bf16(self, rot, rotary=None, q=True, **kw):
        st = word()
        B.locks_rotate_kv(self.q if q else None, self.k, self.v, rot,
                          i32(self.seq), i32(self.pos), i32(self.table),
                          self.qo if q else None, self.kc, self.vc,
                          None if rotary is None else i32(rotary), st, **kw)
        return int(st.item())

    def e4m3(self, rot, rotary=None, q=True, **kw):
        st = word()
        B.locks_rotate_quantise_kv(
            self.q if q else None, self.k, self.v, rot, i32(self.seq),
            i32(self.pos), i32(self.table), self.qo if q else None, self.rec,
            None if rotary is None else i32(rotary), st, **kw)
        return int(st.item())

    def places(self):
        return self.table[self.seq, self.pos // 16], self.pos % 16


def near_bf16(got, want, reach, amplitude=1.0):
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * reach * abs(amplitude) + \
        1e-40
    off = np.abs(got - want) - tol
    assert off.max(initial=-1.0) <= 0, off.max()


def check_bf16(c, freq, axes, pairs, rotary, amplitude=1.0):
    at = [c.pos] if rotary is None else rotary
    for x, got in ((c.q, num(c.qo)), (c.k, num(c.kc)[c.places()[0], :,
                                                     c.places()[1]])):
        x = num(x)
        near_bf16(got, W.rotate(x, at, freq, axes, pairs, amplitude),
                  W.rotate_reach(x, freq, pairs), amplitude)
    phys, slot = c.places()
    assert torch.equal(c.vc[phys, :, slot], c.v.to(torch.bfloat16))
    # nothing else was written
    kept = np.ones((c.P, 16), bool)
    kept[phys, slot] = False
    at = np.nonzero(kept)
    assert (num(c.kc)[at[0], :, at[1]] == 7.0).all()
    assert (num(c.vc)[at[0], :, at[1]] == 9.0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("h_q,h_kv,lens", [(1, 1, [1]), (3, 3, [5, 0, 17]),
                                           (32, 8, [1] * 9), (10, 2, [33, 2]),
                                           (48, 3, [7])])
@pytest.mark.parametrize("dim,pairs", [(128, False), (128, True),
                                       (16, False), (48, True), (96, False)])
def test_rows_into_the_bf16_cache(dtype, h_q, h_kv, lens, dim, pairs):
    c = Case(dim + h_q, lens, h_q, h_kv, dtype)
    freq = frequencies(dim)
    assert c.bf16(B.Rotation(freq, pairs=pairs)) == 0
    check_bf16(c, freq, None, pairs, None)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("pairs", [False, True])
def test_several_axes(axes, pairs):
    c = Case(axes, [20, 3], 8, 2)
    freq = frequencies(128)
    of = [(j * 7) % axes for j in range(64)]
    rotary = c.rng.integers(-50, 5000, (axes, c.n)).astype(np.int32)
    assert c.bf16(B.Rotation(freq, axes=of, pairs=pairs), rotary) == 0
    check_bf16(c, freq, of, pairs, rotary)


def test_amplitude_and_far_positions():
    # positions over the whole of int32: their angles keep every bit
    c = Case(5, [24], 4, 1, "fp32")
    freq = frequencies(128)
    rotary = c.rng.integers(-2 ** 31, 2 ** 31, (1, c.n)).astype(np.int32)
    rotary[0, :4] = [2 ** 31 - 1, -2 ** 31, 0, 131072]
    assert c.bf16(B.Rotation(freq, amplitude=1.25), rotary) == 0
    check_bf16(c, freq, None, False, rotary, 1.25)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("h_q,h_kv,lens", [(1, 1, [1]), (6, 3, [5, 0, 17]),
                                           (32, 8, [1] * 5), (14, 2, [33])])
@pytest.mark.parametrize("dim,pairs", [(128, False), (128, True), (32, False)])
def test_rows_into_the_quantised_cache(dtype, h_q, h_kv, lens, dim, pairs):
    c = Case(dim + h_q, lens, h_q, h_kv, dtype)
    freq = frequencies(dim)
    assert c.e4m3(B.Rotation(freq, pairs=pairs)) == 0
    q = num(c.q)
    near_bf16(num(c.qo), W.rotate(q, [c.pos], freq, None, pairs),
              W.rotate_reach(q, freq, pairs))
    rec = c.rec.cpu().numpy()
    k = num(c.k)
    want, reach = W.rotate(k, [c.pos], freq, None, pairs), \
        W.rotate_reach(k, freq, pairs)
    phys, slot = c.places()
    for i in range(c.n):
        r = rec[phys[i]]
        s = slot[i]
        codes, exps = Q.quantise_rows(num(c.v)[i])
        assert (r[:, 2048 + Q._PLACE[s]] == codes).all()
        assert (r[:, 4112 + s] == exps + 127).all()
        e = r[:, 4096 + s].astype(int) - 127
        top = np.abs(want[i]).max(1)
        slack = 2.0 ** -20 * reach[i].max(1)
        for h in range(c.h_kv):
            assert Q.exponent(top[h] - slack[h]) <= e[h] <= \
                Q.exponent(top[h] + slack[h])
        got = Q.TABLE[r[:, Q._PLACE[s]]] * 2.0 ** e[:, None]
        tol = np.maximum(2.0 ** -4 * np.abs(want[i]),
                         2.0 ** (e[:, None] - 10.0)) + 2.0 ** -20 * reach[i]
        assert (np.abs(got - want[i]) <= tol).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("h_q,h_kv", [(2, 1), (1, 2), (3, 1), (4, 1), (4, 2),
                                      (6, 1)])
@pytest.mark.parametrize("dim,pairs", [(128, False), (64, True)])
def test_few_heads(dtype, h_q, h_kv, dim, pairs):
    """Up to eight rows to a token, as shards of a model have."""
    test_rows_into_the_bf16_cache(dtype, h_q, h_kv, [19, 0, 3], dim, pairs)
    test_rows_into_the_quantised_cache(dtype, h_q, h_kv, [19, 0, 3], dim,
                                       pairs)


def test_without_queries_and_in_place():
    freq = frequencies(128)
    rot = B.Rotation(freq)
    a, b, d = (Case(9, [19, 4], 8, 2) for _ in range(3))
    assert a.bf16(rot) == 0 and b.bf16(rot, q=False) == 0
    assert torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)
    assert (b.qo == 5.0).all()
    # the queries' own memory
    d.q = d.qo = d.q.contiguous()
    assert d.bf16(rot) == 0
    assert torch.equal(a.qo, d.qo)
    e, f = (Case(9, [19, 4], 8, 2) for _ in range(2))
    assert e.e4m3(rot) == 0 and f.e4m3(rot, q=False) == 0
    assert torch.equal(e.rec, f.rec) and torch.equal(e.qo, a.qo)


def test_padding_and_bad_tokens():
    freq = frequencies(128)
    rot = B.Rotation(freq)
    for which in ("bf16", "e4m3"):
        for edit, want in (("pad", 0), ("seq", B.DEV_BAD_PAIR),
                           ("pos", B.DEV_BAD_PAIR), ("far", B.DEV_BAD_PAIR),
                           ("page", B.DEV_BAD_PAGE_ID)):
            c, good = Case(3, [9, 5], 4, 2), Case(3, [9, 5], 4, 2)
            assert getattr(good, which)(rot) == 0
            hit = [2, 11]
            if edit == "pad":
                c.seq[hit] = -1
            elif edit == "seq":
                c.seq[hit] = 2
            elif edit == "pos":
                c.pos[hit] = -1
            elif edit == "far":
                c.pos[hit] = 16 * c.pages
            else:
                c.table[1, 0] = c.P
                hit = [i for i in range(c.n) if c.seq[i] == 1
                       and c.pos[i] < 16]
            assert getattr(c, which)(rot) == want, edit
            rest = [i for i in range(c.n) if i not in hit]
            assert torch.equal(c.qo[rest], good.qo[rest])
            assert (c.qo[hit] == 5.0).all()
            phys, slot = good.places()
            if which == "bf16":
                assert torch.equal(c.kc[phys, :, slot][rest],
                                   good.kc[phys, :, slot][rest])
                assert (c.kc[phys, :, slot][hit] == 7.0).all()
                assert (c.vc[phys, :, slot][hit] == 9.0).all()
            else:
                assert (c.rec[phys[hit], :, 4096 + slot[hit]] == 171).all()


def test_not_a_number_stays_in_its_pair():
    c = Case(4, [3], 2, 1, "fp32")
    c.q[1, 0, 5] = float("nan")
    c.k[2, 0, 70] = float("inf")
    assert c.bf16(B.Rotation(frequencies(128))) == 0
    bad = torch.isnan(c.qo).nonzero().tolist()
    assert bad == [[1, 0, 5], [1, 0, 69]]
    phys, slot = c.places()
    row = c.kc[int(phys[2]), 0, int(slot[2])]
    assert (~torch.isfinite(row)).nonzero().flatten().tolist() == [6, 70]


# ---------------------------------------------------------------------------
# the append of a decode step
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("h_q,h_kv,dim,pairs,axes", [
    (8, 2, 128, False, 1), (8, 2, 128, True, 1), (5, 1, 64, False, 3),
    (48, 16, 96, True, 2), (16, 8, 16, False, 1), (16, 1, 128, False, 4)])
def test_append_is_rotate_then_append(h_q, h_kv, dim, pairs, axes):
    rng = np.random.default_rng(h_q + dim)
    lens = [15, 0, 31, 20, 47]           # three of them fill a page
    batch, pages = len(lens), 4
    freq = frequencies(dim)
    of = [j % axes for j in range(dim // 2)]
    rot = B.Rotation(freq, axes=of, pairs=pairs)
    rotary = None if axes == 1 else i32(
        rng.integers(0, 999, (axes, batch)))
    table = rng.permutation(batch * pages).astype(np.int32).reshape(batch,
                                                                    pages)
    kc = torch.from_numpy(rng.standard_normal(
        (batch * pages, h_kv, 16, 128))).to(torch.bfloat16).to(DEV)
    vc = torch.from_numpy(rng.standard_normal(kc.shape)).to(
        torch.bfloat16).to(DEV)
    q, k, v = (torch.from_numpy(rng.standard_normal((batch, h, 128))).to(
        torch.bfloat16).to(DEV) for h in (h_q, h_kv, h_kv))
    # rotated rows by the other entry point, appended as they are
    kc2, vc2 = kc.clone(), vc.clone()
    q2 = torch.empty_like(q)
    st = word()
    B.locks_rotate_kv(q, k, v, rot, i32(range(batch)), i32(lens), i32(table),
                      q2, kc2, vc2, rotary_positions=rotary, status=st)
    phys = table[np.arange(batch), np.array(lens) // 16]
    k2 = kc2[phys, :, np.array(lens) % 16].contiguous()
    kc2, vc2 = kc.clone(), vc.clone()
    sum2 = B.new_summary_store(batch, h_kv, pages)
    lens2 = i32(lens)
    tau2 = torch.zeros(batch, h_kv, device=DEV)
    B.locks_append_kv(k2, v, kc2, vc2, i32(table), lens2, sum2, tau_out=tau2,
                      status=st)
    lens1, q1 = i32(lens), torch.empty_like(q)
    sum1, tau1 = torch.zeros_like(sum2), torch.zeros_like(tau2)
    B.locks_append_rotated_kv(q, k, v, rot, q1, kc, vc, i32(table), lens1,
                              sum1, rotary_positions=rotary, tau_out=tau1,
                              status=st)
    assert int(st.item()) == 0
    assert torch.equal(q1, q2) and torch.equal(kc, kc2)
    assert torch.equal(vc, vc2) and torch.equal(lens1, lens2)
    assert torch.equal(sum1, sum2) and torch.equal(tau1, tau2)
    assert sum1.any(-1).sum() == 3 * h_kv


def test_append_skips_sequences_that_are_full():
    rot = B.Rotation(frequencies(128))
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = i32([[0, 1], [2, 9]])
    lens = i32([32, 16])
    q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 5.0)
    st = word()
    B.locks_append_rotated_kv(q, k, k, rot, out, kc, vc, table, lens,
                              B.new_summary_store(2, 2, 2), status=st)
    assert int(st.item()) == B.DEV_BAD_SEQ_LEN | B.DEV_BAD_PAGE_ID
    assert (out == 5.0).all() and not kc.any() and lens.tolist() == [32, 16]


def test_decoder_with_a_rotation():
    """Eager and captured steps with unrotated rows give the bytes of a
    decoder that is handed rotated ones."""
    rng = np.random.default_rng(8)
    batch, h_q, h_kv, pages, k = 3, 8, 2, 40, 6
    lens = [500, 333, 590]
    rot = B.Rotation(frequencies(128))
    table = i32(rng.permutation(batch * pages).reshape(batch, pages))
    kc = torch.from_numpy(rng.standard_normal(
        (batch * pages, h_kv, 16, 128))).to(torch.bfloat16).to(DEV)
    vc = torch.randn_like(kc)
    store = B.new_summary_store(batch, h_kv, pages)
    pairs = [(b, p) for b in range(batch) for p in range(lens[b] // 16)]
    B.locks_build_summaries(kc, table, i32([b for b, _ in pairs]),
                            i32([p for _, p in pairs]), store)

    def decoder(**kw):
        return B.LocksDecoder(kc.clone(), vc.clone(), table, store.clone(),
                              h_q, k, seq_lens=i32(lens), append=True, **kw)

    plain, eager = decoder(), decoder(rotation=rot)
    graph = decoder(rotation=rot, graph=True)
    scratch_k, scratch_v = torch.zeros_like(kc), torch.zeros_like(vc)
    for s in range(20):
        q, kn, vn = (torch.from_numpy(rng.standard_normal((batch, h, 128))).to(
            torch.bfloat16).to(DEV) for h in (h_q, h_kv, h_kv))
        at = [n + s for n in lens]
        q2 = torch.empty_like(q)
        B.locks_rotate_kv(q, kn, vn, rot, i32(range(batch)), i32(at), table,
                          q2, scratch_k, scratch_v)
        phys = table[torch.arange(batch, device=DEV),
                     i32(at).long() // 16].long()
        k2 = scratch_k[phys, :, i32(at).long() % 16].contiguous()
        want = [t.clone() for t in plain.step(q2, k_new=k2, v_new=vn)]
        for d in (eager, graph):
            o, lse = d.step(q, k_new=kn, v_new=vn)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), s
            assert torch.equal(d.idx, plain.idx) and d.status() == 0
    for d in (eager, graph):
        assert torch.equal(d.k_cache, plain.k_cache)
        assert torch.equal(d.summaries, plain.summaries)
    with pytest.raises(ValueError):
        graph.step_host(None, None, None, None)


def test_other_stream_and_graph():
    rot = B.Rotation(frequencies(128))
    a, b = Case(11, [40, 9], 8, 2), Case(11, [40, 9], 8, 2)
    assert a.bf16(rot) == 0
    side = torch.cuda.Stream()
    seq, pos, table, st = i32(b.seq), i32(b.pos), i32(b.table), word()
    side.wait_stream(torch.cuda.current_stream())
    args = (b.q, b.k, b.v, rot, seq, pos, table, b.qo, b.kc, b.vc)
    B.locks_rotate_kv(*args, status=st, stream=side)
    side.synchronize()
    assert torch.equal(a.kc, b.kc) and torch.equal(a.qo, b.qo)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.locks_rotate_kv(*args, status=st)
    # another rotation's object may go: the call has copied it
    b.kc.fill_(7.0)
    b.q.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.kc, b.kc)
    near_bf16(num(b.qo), W.rotate(num(b.q), [b.pos], frequencies(128)),
              W.rotate_reach(num(b.q), frequencies(128)))


def test_positions_in_another_order_are_refused():
    """[n][n_axes] instead of [n_axes][n], by all calls and the decoder."""
    c = Case(2, [20, 3], 8, 2)
    rot = B.Rotation(frequencies(128), axes=[j % 3 for j in range(64)])
    wrong = np.zeros((c.n, 3), np.int32)
    for call in (c.bf16, c.e4m3):
        with pytest.raises(ValueError, match="n_axes"):
            call(rot, wrong)
    assert (c.kc == 7.0).all() and (c.rec == 171).all() and (c.qo == 5.0).all()
    lens, q = i32([3, 4]), torch.ones(2, 8, 128, dtype=torch.bfloat16,
                                      device=DEV)
    store = B.new_summary_store(2, 2, c.pages)
    with pytest.raises(ValueError, match="n_axes"):
        B.locks_append_rotated_kv(q, q[:, :2].contiguous(),
                                  q[:, :2].contiguous(), rot, q, c.kc, c.vc,
                                  i32(c.table), lens, store,
                                  rotary_positions=i32(wrong[:2]))
    assert lens.tolist() == [3, 4] and (c.kc == 7.0).all()

    def decoder(**kw):
        return B.LocksDecoder(c.kc, c.vc, i32(c.table), store, 8, 1,
                              seq_lens=lens, **kw)

    for kw in ({"rotation": rot, "rotary_positions": i32(wrong[:2])},
               {"rotation": rot, "rotary_positions": i32(wrong[:3].T.copy())}):
        with pytest.raises(ValueError):
            decoder(append=True, **kw)
    with pytest.raises(ValueError):
        decoder(rotation=rot)
    with pytest.raises(TypeError):
        decoder(append=True, rotation=frequencies(128))
    decoder(append=True, rotation=rot, rotary_positions=i32(np.zeros((3, 2))))


@pytest.mark.parametrize("turned", [False, True])
def test_a_captured_append_leaves_a_full_sequence_alone(turned):
    """A decoder's first captured step, like its eager one, appends to the
    sequences that can take a token, and changes nothing of the others."""
    rng = np.random.default_rng(4)
    batch, h_q, h_kv, pages = 4, 8, 2, 3
    lens = [48, 17, 31, 40]         # full; free; fills a page; a bad page
    table = np.arange(batch * pages).reshape(batch, pages)
    table[3, 2] = batch * pages
    kc = torch.from_numpy(rng.standard_normal(
        (batch * pages, h_kv, 16, 128))).to(torch.bfloat16).to(DEV)
    vc = torch.randn_like(kc)
    rows = [torch.from_numpy(rng.standard_normal((3, batch, h, 128))).to(
        torch.bfloat16).to(DEV) for h in (h_q, h_kv, h_kv)]
    kw = {"rotation": B.Rotation(frequencies(128))} if turned else {}

    def decoder(graph):
        d = B.LocksDecoder(kc.clone(), vc.clone(), i32(table),
                           B.new_summary_store(batch, h_kv, pages), h_q, 2,
                           seq_lens=i32(lens), append=True, graph=graph, **kw)
        for q, k, v in zip(*rows):
            d.step(q, k_new=k, v_new=v)
        return d

    eager, graph = decoder(False), decoder(True)
    assert eager.seq_lens_dev.tolist() == [48, 20, 34, 40]
    assert graph.seq_lens_dev.tolist() == [48, 20, 34, 40]
    for d in (eager, graph):
        assert torch.equal(d.k_cache[:3], kc[:3])
        assert torch.equal(d.v_cache[:3], vc[:3])
    assert torch.equal(graph.k_cache, eager.k_cache)
    assert torch.equal(graph.v_cache, eager.v_cache)
    assert torch.equal(graph.summaries, eager.summaries)
    assert graph.status() == eager.status() == \
        B.DEV_BAD_SEQ_LEN | B.DEV_BAD_PAGE_ID


@pytest.mark.parametrize("h_kv", [1, 16, 20, 21, 22, 27, 32])
def test_append_of_up_to_32_heads(h_kv):
    """Every number of KV heads that the unrotated append takes: bytes of a
    write by hand, summaries of a build of the whole page."""
    rng = np.random.default_rng(h_kv)
    lens, pages = [15, 3, 31], 2
    table = i32(rng.permutation(6).reshape(3, 2))
    kc = torch.from_numpy(rng.standard_normal((6, h_kv, 16, 128))).to(
        torch.bfloat16).to(DEV)
    vc = torch.randn_like(kc)
    k, v = (torch.from_numpy(rng.standard_normal((3, h_kv, 128))).to(
        torch.bfloat16).to(DEV) for _ in range(2))
    want_k, want_v = kc.clone(), vc.clone()
    for b, n in enumerate(lens):
        want_k[table[b, n // 16].long(), :, n % 16] = k[b]
        want_v[table[b, n // 16].long(), :, n % 16] = v[b]
    seq, st = i32(lens), word()
    store, tau = B.new_summary_store(3, h_kv, pages), torch.zeros(
        3, h_kv, device=DEV)
    B.locks_append_kv(k, v, kc, vc, table, seq, store, tau_out=tau, status=st)
    assert int(st.item()) == 0 and seq.tolist() == [16, 4, 32]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    built, tau2 = torch.zeros_like(store), torch.zeros(2, h_kv, device=DEV)
    B.locks_build_summaries(kc, table, i32([0, 2]), i32([0, 1]), built,
                            tau_out=tau2)
    assert torch.equal(store, built) and built[0, :, 0].any(-1).all()
    assert torch.equal(tau[[0, 2]], tau2)
