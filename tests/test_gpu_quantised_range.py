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
