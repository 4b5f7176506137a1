"""The paged cache's attention against its definition, once for each kernel that the sizes
of a call can choose (tests/paged_cases.py; a CPU test checks that the list is complete)."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from paged_cases import BACK, CASES, FRONT, lengths, table_cols, tokens
from test_gpu_paged import World
from w4a16_dequant_gemv_amd import kv

pytestmark = pytest.mark.gpu


def case_id(c):
    return f"d{c.d}-page{c.page}-{c.n_q}on{c.n_kv}-{c.batch}x{c.new}of{c.held}-table{c.limit}-w{c.window}"


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_every_way_the_sizes_choose(case):
    c = case
    held, n = lengths(c)
    w = World(c.batch, c.n_kv, c.d, c.page, seed=c.held + c.new, most=c.limit)
    assert w.cols == table_cols(c) and sum(n) + FRONT + BACK == tokens(c)
    w.append(held)
    for window, sinks in ((c.window, 0), (150, 3)):
        name = kv.attention_config(tokens(c), c.batch, w.cols, c.n_q, c.n_kv, c.d, c.page, window, sinks)
        print(case_id(c), window, name, flush=True)
        x, got = w.attend(n, c.n_q, FRONT, BACK, check=False, window=window, sinks=sinks)
        y = got.cpu().numpy().astype(np.float64)
        assert (y[:FRONT] == 7).all() and (y[len(y) - BACK:] == 7).all()
        weights = {} if "rows_kernel" in name else dict(weights=ref.WEIGHTS_IN_TWO)
        at = FRONT
        for b, (s, m) in enumerate(zip(w.seqs, n)):
            if m:
                o, size, most = ref.attend(s, x[at:at + m], c.d ** -0.5, window, sinks)
                err = np.abs(y[at:at + m] - o)
                tol = ref.tolerance(o, size, most, len(s), c.d, **weights)
                assert bool((err <= tol).all()), (b, float((err / tol).max()), np.argwhere(~(err <= tol))[:3].tolist())
            at += m
    again = w.cache.attend(to_dev(x), w.batch(n, FRONT, ctx=[len(s) - m for s, m in zip(w.seqs, n)]), window=150, sinks=3)
    torch.cuda.synchronize()
    keep = slice(FRONT, len(x) - BACK)
    assert torch.equal(again[keep].view(torch.int16), got[keep].view(torch.int16))      # the same bits again
