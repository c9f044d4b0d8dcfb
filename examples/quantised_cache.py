"""Decoding from the quantised KV cache: one document, many questions.

    python examples/quantised_cache.py

A document's keys and values are written into the 8-bit cache once and stand
at the head of every sequence's page table; each sequence adds its own
question.  Every step writes one token per sequence, then attends twice: over
all tokens, with the document's pages read once for the whole batch
(locks_prefix_decode), and over the k pages that the page summaries select
(locks_score_select, locks_quantised_decode).  The summaries are built from the
keys that pages hold once they are full, read back from the cache
(locks_dequantise_kv), so scores and attention see the same numbers.  Keys,
values and queries are random stand-ins for a model's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_paged_kv_locks_gb300 import binding as B  # noqa: E402


class Server:
    """One layer's cache, summaries and buffers for `batch` sequences that
    share a document of `doc_pages` pages."""

    def __init__(self, batch, h_q, h_kv, doc_pages, max_pages, k,
                 device="cuda"):
        self.h_kv, self.k, self.doc_pages = h_kv, k, doc_pages
        own = max_pages - doc_pages
        P = doc_pages + batch * own
        self.cache = B.new_quantised_cache(P, h_kv, device)
        ids = torch.arange(P, dtype=torch.int32, device=device)
        self.doc = ids[:doc_pages].contiguous()
        self.table = torch.cat([self.doc.expand(batch, -1),
                                ids[doc_pages:].view(batch, own)],
                               1).contiguous()
        self.lens = torch.full((batch,), 16 * doc_pages, dtype=torch.int32,
                               device=device)
        self.host_lens = [16 * doc_pages] * batch
        self.seqs = torch.arange(batch, dtype=torch.int32, device=device)
        self.store = B.new_summary_store(batch, h_kv, max_pages, device)
        self.ws = B.new_workspace(batch, h_q, h_kv, max_pages, k, device)
        self.prefix_ws = B.new_prefix_workspace(batch, h_q, h_kv, max_pages,
                                                doc_pages, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.idx = torch.empty(batch, h_kv, k, dtype=torch.int32,
                               device=device)
        self.outs = [(torch.empty(batch, h_q, 128, dtype=torch.bfloat16,
                                  device=device),
                      torch.empty(batch, h_q, device=device))
                     for _ in range(2)]

    def _ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.lens.device)

    def write_document(self, keys, values):
        """[16 * doc_pages][h_kv][128] rows, once for all sequences."""
        n = 16 * self.doc_pages
        pos = torch.arange(n, dtype=torch.int32, device=keys.device)
        B.locks_quantise_kv(keys, values, torch.zeros_like(pos), pos,
                            self.doc.view(1, -1), self.cache,
                            status=self.status)
        self.summarise([(0, p) for p in range(self.doc_pages)])
        self.store[1:, :, :self.doc_pages] = self.store[:1, :, :self.doc_pages]

    def summarise(self, pairs):
        """Summaries of full pages (sequence, page), from the cache's keys."""
        if not pairs:
            return
        seq, pg = (self._ints(v) for v in zip(*pairs))
        n = len(pairs)
        keys = torch.empty(n, self.h_kv, 16, 128, dtype=torch.bfloat16,
                           device=self.lens.device)
        B.locks_dequantise_kv(self.cache, self.table, seq, pg, keys, None,
                              status=self.status)
        # the n pages as a bf16 cache of their own
        place = torch.zeros_like(self.table)
        place[seq.long(), pg.long()] = torch.arange(
            n, dtype=torch.int32, device=place.device)
        B.locks_build_summaries(keys, place, seq, pg, self.store,
                                status=self.status)

    def write(self, keys, values, counts):
        """counts[b] new tokens of each sequence, rows in sequence order."""
        seq = torch.repeat_interleave(self.seqs, self._ints(counts))
        pos = [self.host_lens[b] + i for b, n in enumerate(counts)
               for i in range(n)]
        B.locks_quantise_kv(keys, values, seq, self._ints(pos), self.table,
                            self.cache, status=self.status)
        full = []
        for b, n in enumerate(counts):
            before = self.host_lens[b] // 16
            self.host_lens[b] += n
            full += [(b, p) for p in range(before, self.host_lens[b] // 16)]
        self.lens += self._ints(counts)
        self.summarise(full)

    def attend_all(self, q):
        o, lse = self.outs[0]
        B.locks_prefix_decode(q, self.cache, self.doc, self.table, self.lens,
                              o, lse, self.prefix_ws)
        return o, lse

    def attend_selected(self, q):
        o, lse = self.outs[1]
        B.locks_score_select(q, self.store, self.lens, self.k, self.idx,
                             self.ws)
        B.locks_quantised_decode(q, self.cache, self.table, self.lens,
                                 self.idx, self.k, o, lse, self.ws)
        return o, lse

    def bad(self):
        """Status bits of all calls so far (0: none)."""
        return int(self.status) | B.locks_read_status(self.ws) | \
            B.locks_read_status(self.prefix_ws)


def main(batch=8, h_q=32, h_kv=8, doc_pages=512, k=64, steps=20, seed=0,
         show=print):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def rows(n, heads):
        return torch.randn(n, heads, 128, generator=gen, device=dev).to(
            torch.bfloat16)

    asked = [3 + 5 * b for b in range(batch)]     # tokens of the questions
    max_pages = doc_pages + (max(asked) + steps + 15) // 16
    s = Server(batch, h_q, h_kv, doc_pages, max_pages, k, dev)
    s.write_document(rows(16 * doc_pages, h_kv), rows(16 * doc_pages, h_kv))
    n = sum(asked)
    s.write(rows(n, h_kv), rows(n, h_kv), asked)
    mass = 0.0
    for _ in range(steps):
        s.write(rows(batch, h_kv), rows(batch, h_kv), [1] * batch)
        q = rows(batch, h_q)
        _, lse_all = s.attend_all(q)
        _, lse_some = s.attend_selected(q)
        # the share of all attention that the selected pages hold
        mass += float(torch.exp(lse_some - lse_all).mean()) / steps
    bf16 = 2 * 2 * 128 * h_kv * 16 * s.cache.shape[0]
    show(f"{batch} sequences of {16 * doc_pages} shared and {asked[0]} to "
         f"{asked[-1]} own tokens, {steps} steps: cache "
         f"{s.cache.numel() / 1e6:.0f} MB (bf16 {bf16 / 1e6:.0f}), {k} of "
         f"{max_pages} pages hold {mass:.3f} of the attention, status "
         f"{s.bad()}")
    return s, mass


if __name__ == "__main__":
    main()
