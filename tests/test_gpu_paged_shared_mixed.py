"""Attention over shared pages in steps that mix single rows with a chunk of a prompt, on both sides
of the average at which a call is run as without shared pages, with tables as wide as a captured step's, and in a
workspace of exactly the stated size."""
import pytest
import torch

from shared_cases import CASES, Case
from test_gpu_paged_shared import Shared, run
from test_gpu_paged_shared_weights import held, kernel_of
from w4a16_dequant_gemv_amd import kv

pytestmark = pytest.mark.gpu

# rows of the chunk, and where it is
MIXED = [(Case(128, 64, 2, 16, ((4, 20),), 700, 1, 0), 100, 0, True), (Case(128, 64, 2, 16, ((4, 20),), 700, 1, 0), 500, 0, False),
         (Case(128, 128, 2, 16, ((2, 30), (1, 9)), 400, 1, 200), 150, 30, True), (Case(64, 64, 2, 8, ((5, 70), (2, 3)), 900, 1, 0), 900, 70, True),
         (Case(64, 64, 4, 16, ((5, 300),), 900, 1, 30), 700, 0, True), (Case(96, 64, 1, 8, ((3, 12),), 300, 1, 0), 90, 11, False),
         (Case(96, 64, 1, 8, ((3, 12),), 300, 1, 0), 70, 11, True),
         (Case(256, 64, 2, 8, ((3, 15), (4, 4)), 300, 1, 0), 200, 17, True), (Case(256, 64, 4, 64, ((3, 90),), 300, 1, 40), 250, 0, True)]


@pytest.mark.parametrize("c,chunk,at,shared", MIXED)
def test_single_rows_and_a_chunk(c, chunk, at, shared):
    w = Shared(c)
    s = w.seqs[at]
    more = chunk - (len(s) - w.pages[0 if at < c.groups[0][1] else 1] * c.page)
    if more > 0:                                               # the chunk is of the sequence's own tokens
        w.append([more if b == at else 0 for b in range(len(w.seqs))])
    n = [chunk if b == at else 1 for b in range(len(w.seqs))]
    name = kernel_of(w, sum(n) + 2, max(w.pages))
    assert ("kv_shared" in name) == shared, name
    x, out, _ = run(w, w.prefix(), n=n, front=1, back=1)
    w.check(x, out, n=n, front=1, weights=held(name))


@pytest.mark.parametrize("c", [c._replace(wide=wide) for c in (CASES[2], CASES[5], CASES[9], CASES[15], CASES[21]) for wide in (60, 1000)])
def test_wide_tables(c):
    w = Shared(c)
    x, out, _ = run(w, w.prefix(), back=2)
    w.check(x, out, weights=held(kernel_of(w, sum(w.new) + 2, max(w.pages))))


@pytest.mark.parametrize("c", CASES)
def test_workspace_of_the_stated_size(c):
    """Nothing is written behind it, and what it holds before does not matter."""
    w = Shared(c)
    T, B, most = sum(w.new), len(w.seqs), max(*w.pages, 1)
    size = kv._shared_workspace_size(T, B, w.table.shape[1], c.page, len(c.groups), most, c.n_q, c.n_kv, c.d)
    room = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    x, out, batch = run(w, w.prefix(), workspace=room[:size])
    assert bool((room[size:] == 0xFF).all())
    w.check(x, out, weights=held(kernel_of(w, T, most)))
