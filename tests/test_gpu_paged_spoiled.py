"""Pages of the paged cache that hold an infinity, a NaN or nothing: who notices.
A row that sees a token of such a page is NaN (or counts zeros); every other row is
what the definition gives, in each of the ways the attention is run."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from test_gpu_paged import World

pytestmark = pytest.mark.gpu

# d, page, n_kv, n_q, sequences besides the first, tokens of the first, its queries, window
WAYS = [
    (64, 64, 2, 4, 0, 400, 300, 0),          # many rows: the page ends inside the call
    (64, 64, 2, 4, 0, 400, 300, 70),
    (128, 128, 2, 16, 0, 700, 400, 100),
    (96, 64, 1, 8, 0, 500, 330, 40),
    (256, 64, 2, 4, 0, 400, 200, 33),
    (256, 64, 1, 1, 20, 300, 150, 0),        # a wide table: runs shared by workgroups
    (128, 64, 1, 1, 9, 300, 200, 50),
    (64, 64, 2, 16, 0, 300, 6, 20),          # few rows whose windows leave the page one after the other
    (128, 64, 2, 4, 0, 300, 10, 20),
    (96, 128, 2, 8, 0, 300, 9, 30),
    (256, 64, 2, 2, 0, 300, 12, 20),
    (64, 64, 8, 64, 150, 200, 5, 20),        # a wave each
]



def run(way, spoil, most=None, seed=0):
    """-> (output, what the definition gives, tolerance, rows x heads that see the page).
    `spoil` changes a page's K and V [page, n_kv, d] in place; the definition is
    computed with that page as `spoil` returns it (K, V)."""
    d, page, n_kv, n_q, others, L, n, window = way
    if n < 20:
        L = L // page * page + 2 * page + 5
        # the middle row is the first that does not see the page
        p = (L - n + n // 2 - window + 1) // page - 1
        L -= (L - n + n // 2 - window + 1) % page
    else:
        p = (L - n) // page + 1
    w = World(1 + others, n_kv, d, page, seed=seed, most=most or 1024)
    k, v = w.values(L, n_kv), w.values(L, n_kv)
    at = slice(p * page, (p + 1) * page)
    clean = k.copy(), v.copy()
    kept = spoil(k[at], v[at])
    clean[0][at], clean[1][at] = kept
    extra = [w.values(30, n_kv) for _ in range(2 * others)]
    gk, gv = (np.concatenate([x] + y) for x, y in ((k, extra[::2]), (v, extra[1::2])))
    w.cache.append(to_dev(gk), to_dev(gv), w.batch([L] + [30] * others))
    w.seqs[0].append(*clean)
    for s, a, b in zip(w.seqs[1:], extra[::2], extra[1::2]):
        s.append(a, b)
    q = [n] + [1] * others
    x = w.values(sum(q), n_q)
    got = w.cache.attend(to_dev(x), w.batch(q, ctx=[len(s) - m for s, m in zip(w.seqs, q)]), window=window)
    torch.cuda.synchronize()
    y = got.cpu().numpy().astype(np.float64)
    want, tol, sees = np.zeros_like(y), np.zeros_like(y), np.zeros(y.shape[:2], bool)
    row = 0
    for i, (s, m) in enumerate(zip(w.seqs, q)):
        o, size, most_score = ref.attend(s, x[row:row + m], d ** -0.5, window)
        want[row:row + m], tol[row:row + m] = o, ref.tolerance(o, size, most_score, len(s), d)
        row += m
    for i in range(n):
        first = max(0, L - n + i - window + 1) if window else 0
        sees[i] = first < (p + 1) * page and L - n + i >= p * page
    assert sees.any() and not sees.all()
    return y, want, tol, sees, (w, p)


def check(y, want, tol, right):
    err = np.abs(y - want)
    ok = err[right] <= tol[right]
    assert bool(ok.all()), np.argwhere(right & ~(err <= tol).all(-1))[:5].tolist()


@pytest.mark.parametrize("most", [1024, 8192])
@pytest.mark.parametrize("which", ["v", "k"])
@pytest.mark.parametrize("way", WAYS)
def test_an_infinity_in_a_finished_page(way, which, most):
    """One infinite value of kv head 0: its page's scale is infinite, so every token of
    the page is spoiled for that head's queries, and nothing else is."""
    def spoil(k, v):
        kept = k.copy(), v.copy()
        (v if which == "v" else k)[17, 0, 5] = -np.inf
        return kept
    y, want, tol, sees, _ = run(way, spoil, most)
    group = way[3] // way[2]
    bad = sees.copy()
    bad[:, group:] = False
    assert np.isnan(y[bad]).all()
    check(y, want, tol, ~bad)


@pytest.mark.parametrize("most", [1024, 8192])
@pytest.mark.parametrize("way", WAYS)
def test_a_page_with_zero_scales(way, most):
    """A listed page that nobody filled (the pool begins with zeros for scales): its
    tokens are zeros, scores and values, for the rows that see it."""
    d, page, n_kv, n_q, others, L, n, window = way
    y, _, _, _, (w, p) = run(way, lambda k, v: (k.copy(), v.copy()), most)
    at = int(w.table[0, p])
    w.cache.k_scale[at] = 0
    w.cache.v_scale[at] = 0
    s = w.seqs[0]
    s.k[p * page:(p + 1) * page] = 0
    s.v[p * page:(p + 1) * page] = 0
    w.attend([n] + [1] * others, n_q, window=window)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d,page,steps,at", [
    (64, 64, [30, 40], 10),              # in the ring when the page fills
    (64, 64, [30, 40], 50),              # in the call that fills it
    (128, 128, [300], 200),              # in a page of new tokens only
    (96, 128, [127, 1], 127),            # the token that fills it
    (256, 64, [60, 70], 63),
    (128, 256, [256], 0),
])
def test_a_bad_value_in_a_page_that_becomes_full(d, page, steps, at, which, bad):
    """The page's scale says so, and every row that sees the page is NaN; the other
    head, K or V, and the other pages are what they are without it."""
    n_kv, total = 2, sum(steps)
    w = World(1, n_kv, d, page, seed=d + at)
    k, v = w.values(total, n_kv), w.values(total, n_kv)
    x = k if which == "k" else v
    x[at, 1, d // 2] = bad
    done = 0
    for n in steps:
        w.cache.append(to_dev(k[done:done + n]), to_dev(v[done:done + n]), w.batch([n], ctx=[done]))
        done += n
    torch.cuda.synchronize()
    ks, vs = w.cache.k_scale.cpu().numpy(), w.cache.v_scale.cpu().numpy()
    for p in range(total // page):
        for name, y, scale in (("k", k, ks), ("v", v, vs)):
            for h in range(n_kv):
                with np.errstate(invalid="ignore"):
                    got, want = scale[w.table[0, p], h], ref.quantize(y[p * page:(p + 1) * page, h])[1]
                if name == which and h == 1 and p == at // page:
                    assert np.isnan(got) if np.isnan(bad) else np.isinf(got)
                else:
                    assert got == want, (p, name, h)
    pages = w.cache.read(to_dev(w.table[0, :1].copy()))["kv".index(which)]
    if at < page and np.isnan(bad):
        assert torch.isnan(pages[0, 1]).all()
    assert torch.isfinite(pages[0, 0]).all()
    w.seqs[0].append(*(np.where(np.isfinite(y), y, 0).astype(np.float16) for y in (k, v)))
    q = w.values(1, 4)
    y = w.cache.attend(to_dev(q), w.batch([1], ctx=[total - 1])).cpu().numpy()
    o, size, most = ref.attend(w.seqs[0], q, d ** -0.5)
    assert np.isnan(y[:, 2:]).all()
    assert bool((np.abs(y - o) <= ref.tolerance(o, size, most, total, d))[:, :2].all())
    # windows that have left the page
    left = total - (at // page + 1) * page
    if left > 1:
        y = w.cache.attend(to_dev(q), w.batch([1], ctx=[total - 1]), window=left).cpu().numpy()
        o, size, most = ref.attend(w.seqs[0], q, d ** -0.5, left)
        assert bool((np.abs(y - o) <= ref.tolerance(o, size, most, total, d)).all())


def test_positions_outside_the_table_stay_nan():
    """A key that was rotated to a position outside the table is NaN in the ring, and
    so is what sees it there; once its page is full, all that see the page."""
    d, page = 64, 64
    w = World(1, 1, d, page, seed=3)
    table = ref.rope_table(40, d)
    x = w.values(70, 2)
    positions = (np.arange(70) % 40).astype(np.int32)
    positions[33] = 40
    k, v = (np.ascontiguousarray(x[:, i:i + 1]) for i in range(2))
    for lo, hi in ((0, 50), (50, 70)):
        w.cache.append(to_dev(k[lo:hi]), to_dev(v[lo:hi]), w.batch([hi - lo], ctx=[lo]), rope=to_dev(table),
                       positions=to_dev(positions[lo:hi].copy()))
        q = to_dev(w.values(hi - lo, 2))
        y = w.cache.attend(q, w.batch([hi - lo], ctx=[lo]))
        sees = torch.arange(lo, hi, device="cuda") >= (33 if lo == 0 else 0)
        assert torch.isnan(y[sees]).all() and torch.isfinite(y[~sees]).all()
        y = w.cache.attend(q[-1:], w.batch([1], ctx=[hi - 1]), window=6)
        assert torch.isfinite(y).all()
