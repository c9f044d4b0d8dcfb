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
