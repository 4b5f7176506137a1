"""Attention over the paged cache with scores of any size: queries and keys are small
whole numbers, so that scores are exact, and far enough apart that each row's output is
the value of its best token."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from test_gpu_paged import World

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale,times", [(100.0, 1), (3e5, 1), (1e6, 1), (1e6, 2048), (0.125, 2048)])
@pytest.mark.parametrize("d,page,n_kv,n_q,held,n,window", [
    (64, 64, 2, 8, [500], [300], 0),         # many rows of a sequence
    (128, 128, 1, 8, [700], [400], 100),
    (96, 64, 1, 4, [500], [400], 3),         # windows whose scores may all be negative
    (256, 64, 1, 2, [300], [200], 0),
    (128, 128, 2, 2, [300, 900], [1, 3], 0),     # few rows
    (64, 64, 1, 8, [700, 130], [5, 4], 3),
    (256, 64, 1, 4, [900], [2], 0),
])
@pytest.mark.parametrize("most", [1024, 16384])
def test_the_best_token_takes_all(d, page, n_kv, n_q, held, n, window, scale, times, most):
    w = World(len(held), n_kv, d, page, seed=d + times, most=most)
    T = sum(held)
    k = w.rng.integers(-20, 21, (T, n_kv, d))
    k[:, :, 0] = 0
    at = 0
    for L in held:                                       # every page's scale is 1: its codes are the keys
        k[at:at + L:16, :, 0] = 127
        at += L
    k = k.astype(np.float16)
    v = w.values(T, n_kv)
    w.cache.append(to_dev(k), to_dev(v), w.batch(held))
    at = 0
    for s, L in zip(w.seqs, held):
        s.append(k[at:at + L], v[at:at + L])
        at += L
    q = w.rng.integers(-20, 21, (sum(n), n_q, d)) * times
    q[:, :, 0] = 0                                       # the column of 127 does not count
    q = q.astype(np.float16)
    y = w.cache.attend(to_dev(q), w.batch(n, ctx=[L - m for L, m in zip(held, n)]), scale=scale, window=window)
    torch.cuda.synchronize()
    y = y.cpu().numpy().astype(np.float64)
    at, clear, group = 0, 0, n_q // n_kv
    for s, m in zip(w.seqs, n):
        o, size, _ = ref.attend(s, q[at:at + m], scale, window)
        tol = ref.tolerance(o, size, 0.0, len(s), d)
        ok = np.isfinite(y[at:at + m]).all(-1)
        assert ok.all(), np.argwhere(~ok)[:3].tolist()
        for h in range(n_q):
            kh = s.values(h // group)[0]
            score = q[at:at + m, h].astype(np.float64) @ kh.T
            i, j = len(s) - m + np.arange(m)[:, None], np.arange(len(s))[None]
            score[(j > i) | ((i - j >= window) if window else False)] = -np.inf
            best = np.sort(score, 1)
            # the runner-up is 2^30 times lighter, with the scores' own rounding in binary32 allowed for
            gap = (best[:, -1] - best[:, -2]) * scale * np.log2(np.e)
            sure = gap >= 30 + np.abs(best[:, -1]) * scale * 2.0**-21
            clear += int(sure.sum())
            assert bool((np.abs(y[at:at + m, h] - o[:, h]) <= tol[:, h])[sure].all()), h
        at += m
    assert clear >= sum(n) * n_q * 3 // 4


@pytest.mark.parametrize("d,page,tokens,others,most", [
    (64, 64, 330, 0, 512),                   # a row block a workgroup
    (128, 128, 330, 0, 512),
    (96, 64, 200, 0, 512),
    (256, 64, 200, 0, 512),
    (64, 64, 330, 0, 16384),                 # runs shared by workgroups
    (128, 128, 330, 1, 16384),
    (96, 128, 300, 2, 16384),
    (256, 128, 300, 0, 16384),
    (64, 64, 200, 300, 256),                 # a wave each
])
def test_few_rows_have_their_weights_in_full(d, page, tokens, others, most):
    """With few rows a sequence a weight is two fp16 parts: far below one part's rounding."""
    n_kv = 8
    w = World(1 + others, n_kv, d, page, seed=d, most=most)
    k, v, q, scale = ref.balanced(n_kv, d, tokens)
    T = tokens + 3 * others
    extra = w.values(T - tokens, n_kv), w.values(T - tokens, n_kv)
    w.cache.append(to_dev(np.concatenate([k, extra[0]])), to_dev(np.concatenate([v, extra[1]])), w.batch([tokens] + [3] * others))
    w.seqs[0].append(k, v)
    x = np.concatenate([q, w.values(others, n_kv)])
    y = w.cache.attend(to_dev(x), w.batch([1] * (1 + others), ctx=[tokens - 1] + [2] * others), scale=scale)
    torch.cuda.synchronize()
    o, size, top = ref.attend(w.seqs[0], q, scale)
    tol = ref.tolerance(o, size, top, tokens, 0, ref.WEIGHTS_IN_TWO)
    err = np.abs(y[:1].cpu().numpy().astype(np.float64) - o)
    assert bool((err <= tol).all()), float((err / tol).max())
