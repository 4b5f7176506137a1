"""Attention over the paged cache for sequences that share their first pages, against the
definition in 64 bits of each sequence for itself."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from shared_cases import Case, lengths, sizes
from test_gpu_paged import World
from w4a16_dequant_gemv_amd import W4A16Error, kv

pytestmark = pytest.mark.gpu


def i32(v):
    return to_dev(np.ascontiguousarray(v, np.int32))


class Shared(World):
    """Groups of sequences over the same first pages, each with tokens of its own behind them."""

    def __init__(self, c, seed=0, own=None):
        owns, self.new = lengths(c)
        owns = owns if own is None else own
        T, B, cols, G, most = sizes(c)
        super().__init__(B, c.n_kv, c.d, c.page, most=(cols + 2) * c.page, seed=seed)
        self.cols = cols
        self.table = self.table[:, :cols].copy()
        self.c, self.cu = c, np.concatenate([[0], np.cumsum([n for _, n in c.groups])])
        self.pages = [p for p, _ in c.groups]
        for g, p in enumerate(self.pages):
            lo, hi = self.cu[g], self.cu[g + 1]
            k, v = self.values(p * c.page, c.n_kv), self.values(p * c.page, c.n_kv)
            one = lambda x, b: np.ascontiguousarray(x[b:b + 1])
            if p:
                self.cache.append(to_dev(k), to_dev(v), kv.PagedBatch(i32([0, len(k)]), i32([0]), i32(one(self.table, lo)),
                                                                    i32(self.slots[lo:lo + 1])))
            for b in range(lo, hi):
                self.table[b, :p] = self.table[lo, :p]
                self.seqs[b].append(k, v)
        self.append(owns)

    def prefix(self, pages=None, max_pages=None, cu=None):
        return kv.SharedPrefix(i32(self.cu if cu is None else cu), i32(self.pages if pages is None else pages),
                               max(self.pages) if max_pages is None else max_pages)

    def held(self, n=None):
        return [len(s) - m for s, m in zip(self.seqs, self.new if n is None else n)]

    def check(self, x, out, n=None, front=0, scale=None, hidden=None, weights=2.0**-11, skip=()):
        y = out.cpu().numpy().astype(np.float64)
        at = front
        assert (y[:front] == 7).all()
        for b, (s, m) in enumerate(zip(self.seqs, self.new if n is None else n)):
            if b in skip:
                assert (y[at:at + m] == 7).all(), b
            elif m:
                o, size, most = ref.attend(s, x[at:at + m], self.d ** -0.5 if scale is None else scale, hidden=hidden[b] if hidden else ())
                err, tol = np.abs(y[at:at + m] - o), ref.tolerance(o, size, most, len(s), self.d, weights=weights)
                assert bool((err <= tol).all()), (b, float((err / tol).max()), np.argwhere(~(err <= tol))[:3].tolist())
            at += m
        assert (y[at:] == 7).all()


def run(w, prefix, n=None, front=0, back=0, seed=1, **kw):
    n = w.new if n is None else n
    w.rng = np.random.default_rng(seed)
    x = w.values(sum(n) + front + back, w.c.n_q)
    out = torch.full(x.shape, 7.0, dtype=torch.float16, device="cuda")
    batch = w.batch(n, front, ctx=w.held(n))
    w.cache.attend(to_dev(x), batch, out=out, prefix=prefix, **kw)
    torch.cuda.synchronize()
    return x, out, batch


SMALL = [
    Case(128, 128, 2, 8, ((3, 5),), 200, 1, 0),
    Case(64, 64, 2, 2, ((1, 1),), 3, 1, 0),
    Case(64, 64, 1, 8, ((7, 20), (2, 3), (1, 1)), 150, 1, 0),
    Case(128, 64, 8, 8, ((9, 40),), 100, 1, 0),
    Case(96, 64, 2, 8, ((4, 6), (5, 9)), 90, 5, 0),
    Case(256, 64, 2, 16, ((5, 7),), 130, 3, 0),
    Case(128, 256, 1, 40, ((2, 9),), 300, 1, 3),
    Case(128, 128, 2, 16, ((4, 3),), 400, 60, 0),
    Case(64, 128, 2, 8, ((6, 2), (3, 2)), 900, 300, 0),
    Case(256, 128, 1, 4, ((3, 4),), 300, 90, 0),
]


@pytest.mark.parametrize("c", SMALL)
def test_against_the_definition(c):
    w = Shared(c)
    x, out, batch = run(w, w.prefix(), front=2, back=3)
    w.check(x, out, front=2)
    again = torch.full_like(out, 7.0)
    w.cache.attend(to_dev(x), batch, out=again, prefix=w.prefix())
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
