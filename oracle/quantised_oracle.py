"""Plain float64 CPU statement of the quantised KV cache and its attention.

TEST INFRASTRUCTURE ONLY, like locks_oracle.py: nothing in the product path
imports it, and it shares no code with the CUDA library.  The record format is
the one that include/locks.h describes; the attention is the textbook softmax
over the numbers that the records stand for, computed token by token position.
"""
from __future__ import annotations

import math

import numpy as np

PAGE, DIM, RECORD = 16, 128, 4128
E_LO, E_HI = -32, 31


def e4m3_table() -> np.ndarray:
    """The number of each code: sign, 4 exponent bits (bias 7), 3 fraction
    bits; exponent and fraction all ones is NaN."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            a = math.nan
        t[c] = -a if c & 0x80 else a
    return t


TABLE = e4m3_table()


def exponent(absmax: float) -> int:
    """Least e with absmax <= 448 * 2^e, within the limits."""
    for e in range(E_LO, E_HI):
        if absmax <= 448.0 * 2.0 ** e:
            return e
    return E_HI


def quantise_rows(x: np.ndarray):
    """rows [n][128] -> (codes [n][128] uint8 in dim order, exponents [n])."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.shape, np.uint8)
    exps = np.zeros(x.shape[0], np.int64)
    size = TABLE[:127]
    for i, row in enumerate(x):
        top = np.max(np.abs(row[~np.isnan(row)]), initial=0.0)
        e = exps[i] = exponent(top)
        mag = np.minimum(np.abs(row) / 2.0 ** e, 448.0)
        lo = np.clip(np.searchsorted(size, mag, side="right") - 1, 0, 125)
        below, above = mag - size[lo], size[lo + 1] - mag
        up = (above < below) | ((above == below) & (lo % 2 == 1))
        c = (lo + up).astype(np.uint8) | (np.signbit(row) << 7).astype(np.uint8)
        codes[i] = np.where(np.isnan(row), 0x7F, c)
    return codes, exps


def byte_of(slot: int, d: int) -> int:
    """Place of dim d of a row in slot `slot` among the row codes."""
    c = (d // 16) ^ (slot & 6) ^ (5 if slot & 1 else 0)
    return 128 * slot + 16 * c + d % 16


_PLACE = np.array([[byte_of(s, d) for d in range(DIM)] for s in range(PAGE)])


def write(cache, k, v, seq_ids, positions, page_table):
    """k, v [n][h_kv][128] into the cache [P][h_kv][4128] (in place)."""
    for i, (b, pos) in enumerate(zip(seq_ids, positions)):
        if b < 0:
            continue
        rec = cache[page_table[b, pos // PAGE]]
        s = pos % PAGE
        for part, x in ((0, k), (1, v)):
            codes, e = quantise_rows(x[i])
            rec[:, 2048 * part + _PLACE[s]] = codes
            rec[:, 4096 + 16 * part + s] = e + 127


def read(rec):
    """records [..., 4128] -> keys, values [..., 16, 128] float64."""
    out = []
    for part in (0, 1):
        codes = rec[..., 2048 * part + _PLACE]
        e = rec[..., 4096 + 16 * part:4112 + 16 * part].astype(np.float64) - 127
        out.append(TABLE[codes] * np.exp2(e)[..., None])
    return out


def attend(q, K, V):
    """q [G][128], K, V [T][128] -> (o [G][128], lse [G], mass [G][128]),
    mass = sum softmax |v|, the scale of an output's error."""
    G = q.shape[0]
    if K.shape[0] == 0:
        return np.zeros((G, DIM)), np.full(G, -np.inf), np.zeros((G, DIM))
    x = q @ K.T / math.sqrt(DIM)
    top = x.max(axis=1, keepdims=True)
    w = np.exp(x - top)
    total = w.sum(axis=1, keepdims=True)
    p = w / total
    return p @ V, (top + np.log(total))[:, 0], p @ np.abs(V)


def tokens(cache, table_row, h, pages, length, prefix=None):
    """Valid tokens of the listed pages of one sequence and head."""
    pages = np.asarray(list(pages), np.int64)
    pages = pages[(pages >= 0) & (PAGE * pages < length)]
    phys = np.array([prefix[p] if prefix is not None and p < len(prefix)
                     else table_row[p] for p in pages], np.int64)
    K, V = read(cache[phys, h].reshape(-1, RECORD))
    keep = (PAGE * pages[:, None] + np.arange(PAGE) < length).reshape(-1)
    return K.reshape(-1, DIM)[keep], V.reshape(-1, DIM)[keep]


def decode(q, cache, page_table, seq_lens, idx=None, prefix=None):
    """(o, lse, mass) [batch][h_q].. over listed pages idx [batch][h_kv][k],
    or every page; `prefix`: physical pages that take the place of the first
    entries of every table."""
    batch, h_q, _ = q.shape
    h_kv = cache.shape[1]
    G = h_q // h_kv
    o = np.zeros((batch, h_q, DIM))
    lse = np.zeros((batch, h_q))
    mass = np.zeros((batch, h_q, DIM))
    for b in range(batch):
        L = int(seq_lens[b])
        for h in range(h_kv):
            pages = range(-(-L // PAGE)) if idx is None else \
                [int(p) for p in idx[b, h]]
            K, V = tokens(cache, page_table[b], h, pages, L, prefix)
            sl = slice(h * G, (h + 1) * G)
            o[b, sl], lse[b, sl], mass[b, sl] = attend(q[b, sl], K, V)
    return o, lse, mass
