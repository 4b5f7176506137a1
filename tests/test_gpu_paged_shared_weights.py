"""Attention over shared pages gives what the same call without them gives, but for the order of
sums: weights are held in two fp16 parts whichever kernel takes the shared pages, also where one
part's rounding would show (half of the tokens nearly cancel the other half)."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from shared_cases import CASES, Case, sizes
from test_gpu_paged_shared import KINDS, Shared, run
from w4a16_dequant_gemv_amd import kv

pytestmark = pytest.mark.gpu


def kernel_of(w, T, most):
    c = w.c
    return kv.attention_config(T, len(w.seqs), w.table.shape[1], c.n_q, c.n_kv, c.d, c.page, groups=len(c.groups), max_pages=most)


def held(name):
    """A call that is run as without shared pages keeps its weights as that does."""
    return 2.0**-11 if "kv_attend_rows" in name else ref.WEIGHTS_IN_TWO


# d, page, n_kv, n_q, (shared pages, sequences), own, rows of a sequence
BALANCED = [Case(128, 64, 8, 64, ((6, 400),), 8, 1, 0), Case(128, 128, 8, 64, ((3, 64),), 8, 1, 0), Case(64, 64, 8, 64, ((6, 400),), 8, 1, 0),
            Case(96, 64, 8, 64, ((6, 400),), 8, 1, 0), Case(256, 64, 8, 64, ((3, 300),), 8, 1, 0), Case(128, 64, 8, 16, ((5, 5),), 8, 1, 0),
            Case(64, 64, 8, 8, ((5, 7),), 8, 1, 0), Case(96, 64, 8, 8, ((4, 30),), 8, 1, 0), Case(256, 64, 8, 8, ((5, 4),), 8, 1, 0)]


@pytest.mark.parametrize("c", BALANCED)
def test_weights_in_two_parts(c):
    """Every sequence has the same tokens: the shared pages' and 6 to 8 more; so every row of a head has to be the same."""
    p, B = c.groups[0]
    w = Shared(c)
    k, v, q, scale = ref.balanced(c.n_kv, c.d, p * c.page + 8)
    shared = p * c.page
    # written over what is there
    i32 = lambda x: to_dev(np.ascontiguousarray(x, np.int32))
    w.cache.append(to_dev(k[:shared]), to_dev(v[:shared]),
                   kv.PagedBatch(i32([0, shared]), i32([0]), i32(w.table[:1]), i32(w.slots[:1])))
    own = np.array([6 + b % 3 for b in range(B)])
    rows = np.concatenate([np.arange(shared, shared + n) for n in own])
    w.cache.append(to_dev(k[rows]), to_dev(v[rows]), w.batch(own.tolist(), ctx=[shared] * B))
    x = np.repeat(np.repeat(q, c.n_q // c.n_kv, 1), B, 0)
    batch = w.batch([1] * B, ctx=shared + own - 1)
    name = kernel_of(w, B, p)
    assert "kv_shared" in name
    y = w.cache.attend(to_dev(x), batch, scale=scale, prefix=w.prefix())
    torch.cuda.synchronize()
    y = y.cpu().numpy().astype(np.float64)
    for n in (6, 7, 8):
        s = ref.Sequence(c.n_kv, c.d, c.page)
        s.append(k[:shared + n], v[:shared + n])
        o, size, top = ref.attend(s, x[:1], scale)
        tol = ref.tolerance(o, size, top, len(s), 0, ref.WEIGHTS_IN_TWO)      # scores are exact: no products' roundings
        worst = float((np.abs(y[own == n] - o) / tol).max())
        assert worst <= 1, (name, n)


@pytest.mark.parametrize("c", CASES)
def test_every_kernel(c):
    w = Shared(c)
    x, out, _ = run(w, w.prefix(), front=2, back=3)
    w.check(x, out, front=2, weights=held(kernel_of(w, sum(w.new) + 5, max(*w.pages, 1))))


@pytest.mark.parametrize("c", KINDS)
def test_groups_that_change(c):
    """Fewer pages named than are shared, sequences that no group names, a cap below what is shared."""
    for kw in (dict(pages=[1, 2, 1]), dict(cu=[1, 3, 3, 5]), dict(max_pages=2)):
        w = Shared(c)
        x, out, _ = run(w, w.prefix(**kw), front=1, back=1)
        most = kw.get("max_pages", max(w.pages))
        w.check(x, out, front=1, weights=held(kernel_of(w, sum(w.new) + 2, most)))


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    rng = np.random.default_rng(900 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]
    n_kv, group = pick((1, 8), (2, 4), (4, 1), (3, 7), (8, 8), (1, 40))
    page = pick(64, 128, 256)
    groups = tuple((int(rng.integers(0, 1 + 900 // page)), int(rng.integers(1, pick(3, 12, 90)))) for _ in range(pick(1, 1, 2, 4)))
    c = Case(pick(64, 96, 128, 256), page, n_kv, n_kv * group, groups, int(rng.integers(1, pick(60, 400, 1500))), pick(1, 1, 1, 3), pick(0, 0, 9))
    w = Shared(c, seed=seed)
    name = kernel_of(w, sizes(c)[0] + 3, max(*w.pages, 1))
    print(seed, c, name, flush=True)
    x, out, batch = run(w, w.prefix(), front=3, seed=seed)
    w.check(x, out, front=3, weights=held(name))
    again = torch.full_like(out, 7.0)
    w.cache.attend(to_dev(x), batch, out=again, prefix=w.prefix())
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
