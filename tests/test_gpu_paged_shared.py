"""Attention over the paged cache for sequences that share their first pages, against the
definition in 64 bits of each sequence for itself."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from shared_cases import CASES, Case, lengths, sizes
from test_gpu_paged import World
from w4a16_dequant_gemv_amd import W4A16Error, kv

pytestmark = pytest.mark.gpu


def i32(v):
    return to_dev(np.ascontiguousarray(v, np.int32))


class Shared(World):
    """Groups of sequences over the same first pages, each with tokens of its own behind them."""

    def __init__(self, c, seed=0, own=None, pool=None):
        owns, self.new = lengths(c)
        owns = owns if own is None else own
        T, B, cols, G, most = sizes(c)
        super().__init__(B, c.n_kv, c.d, c.page, pool=pool, most=(cols + 2) * c.page, seed=seed)
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
                               max(*self.pages, 1) if max_pages is None else max_pages)

    def held(self, n=None):
        return [len(s) - m for s, m in zip(self.seqs, self.new if n is None else n)]

    def check(self, x, out, n=None, front=0, scale=None, hidden=None, weights=2.0**-11, skip=()):
        y = out.cpu().numpy().astype(np.float64)
        at = front
        assert (y[:front] == 7).all()
        # of many sequences the first ones, those at the groups' borders, the last one and some
        some = {*range(6), *self.cu.tolist(), *(self.cu - 1).tolist(), *np.random.default_rng(1).integers(0, len(self.seqs), 16).tolist()}
        for b, (s, m) in enumerate(zip(self.seqs, self.new if n is None else n)):
            assert np.isfinite(y[at:at + m]).all(), b
            if b in skip:
                assert (y[at:at + m] == 7).all(), b
            elif m and b in some:
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


def weights(c):
    """How the kernel that the sizes choose keeps its weights: one fp16 value where it takes many rows."""
    T, B, cols, G, most = sizes(c)
    name = kv.attention_config(T + 5, B, cols, c.n_q, c.n_kv, c.d, c.page, groups=G, max_pages=max(most, 1))
    return 2.0**-11 if "true" in name or "rows" in name else ref.WEIGHTS_IN_TWO


@pytest.mark.parametrize("c", CASES)
def test_against_the_definition(c):
    w = Shared(c)
    x, out, batch = run(w, w.prefix(), front=2, back=3)
    w.check(x, out, front=2, weights=weights(c))
    again = torch.full_like(out, 7.0)
    w.cache.attend(to_dev(x), batch, out=again, prefix=w.prefix())
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


# one kernel of each kind, with three groups of which the last has one sequence
KINDS = [Case(128, 64, 2, 8, ((5, 6), (3, 4), (2, 1)), 150, 1, 0), Case(64, 64, 4, 64, ((6, 150), (5, 109), (2, 1)), 60, 1, 8),
         Case(256, 64, 4, 64, ((6, 100), (5, 100), (4, 1)), 60, 1, 0)]


@pytest.mark.parametrize("c", KINDS)
@pytest.mark.parametrize("what", ["fewer", "more", "some", "none", "capped", "nobody", "shorter"])
def test_what_is_shared(c, what):
    """Fewer pages named than are shared; a cap below them; sequences that no group names; groups without sequences; sequences
    (the first among them) that end inside the shared pages: the result is every sequence's own either way."""
    w = Shared(c)
    kw = dict(fewer=dict(pages=[p // 2 for p in w.pages]), more=dict(pages=[1 << 30] * 3, max_pages=min(w.pages)),
              some=dict(cu=[1, 3, 3, 5], pages=[w.pages[0], 7, w.pages[0] - 1]), none=dict(pages=[0, 0, -5]), capped=dict(max_pages=2),
              nobody=dict(cu=[0, 0, 0, 0]), shorter={})[what]
    if what == "shorter":                                      # whole pages, so that none is read from the ring
        for b, pages in ((0, 1), (2, 2), (5, w.pages[0])):
            s = w.seqs[b]
            s.k, s.v = s.k[:pages * c.page], s.v[:pages * c.page]
    x, out, _ = run(w, w.prefix(**kw), front=1, back=1)
    w.check(x, out, front=1)


@pytest.mark.parametrize("c", KINDS)
def test_skipped_sequences_and_sequences_without_rows(c):
    """A group's first sequence is skipped (its block table and length hold anything), or has no rows; so does another one."""
    for how in ("length", "slot", "rows"):
        w = Shared(c)
        n, skip = list(w.new), (0, 4)
        ctx, slots, table = w.held(), w.slots.copy(), w.table.copy()
        for b in skip:
            table[b] = -7
            if how == "length":
                ctx[b] = -1
            elif how == "slot":
                slots[b] = len(slots) + 2
            else:
                n[b], ctx[b] = 0, 1 << 29
        w.rng = np.random.default_rng(5)
        x = w.values(sum(n), c.n_q)
        out = torch.full(x.shape, 7.0, dtype=torch.float16, device="cuda")
        w.cache.attend(to_dev(x), w.batch(n, ctx=ctx, slots=slots, table=table), out=out, prefix=w.prefix())
        w.check(x, out, n=n, skip=skip)


@pytest.mark.parametrize("c", KINDS)
def test_pages_that_are_not_there(c):
    w = Shared(c)
    lo, hi = w.cu[0], w.cu[1]
    w.table[lo:hi, 1] = -1                                     # a shared page of the first group
    w.table[w.cu[1]:w.cu[2], 0] = w.cache.pool_pages           # and one of the second
    hidden = [(1,) if b < hi else (0,) if b < w.cu[2] else () for b in range(len(w.seqs))]
    x, out, _ = run(w, w.prefix())
    w.check(x, out, hidden=hidden)


@pytest.mark.parametrize("c", KINDS)
@pytest.mark.parametrize("value", [np.inf, np.nan])
def test_spoiled_pages(c, value):
    """The scale that a shared page gets from an infinity or NaN: NaN in its group's rows of that kv head, in no others."""
    w = Shared(c)
    g, h = 1, c.n_kv - 1
    page = int(w.table[w.cu[g], 1])
    for scale in (w.cache.k_scale, w.cache.v_scale):
        w2 = scale[page, h].clone()
        scale[page, h] = float(value)
        x, out, _ = run(w, w.prefix())
        scale[page, h] = w2
        y = out.cpu().numpy()
        mine, heads = slice(w.cu[g], w.cu[g + 1]), slice(h * c.n_q // c.n_kv, (h + 1) * c.n_q // c.n_kv)
        assert np.isnan(y[mine, heads]).all()
        y[mine, heads] = 0
        assert np.isfinite(y).all()


def test_large_and_small_scores():
    """Scores whose weights leave binary32's range if taken from the wrong maximum, in the shared part, in the own part, in both."""
    c = Case(128, 64, 2, 8, ((4, 5),), 150, 1, 0)
    for big in ("shared", "own", "both"):
        w = Shared(c)
        for scale in (w.cache.k_scale,):
            ids = torch.from_numpy(w.table[0, :4].astype(np.int64)).cuda()
            if big in ("shared", "both"):
                scale[ids] *= 64
        for s in w.seqs:
            if big in ("shared", "both"):
                s.k[:256] *= np.float16(64)
        if big in ("own", "both"):
            w.cache.k_tail *= 64
            own = torch.from_numpy(np.unique(w.table[:, 4:])).long().cuda()
            w.cache.k_scale[own] *= 64
            for s in w.seqs:
                s.k[256:] *= np.float16(64)
        for sc in (w.d ** -0.5, 3.0):
            x, out, _ = run(w, w.prefix(), scale=sc)
            w.check(x, out, scale=sc, weights=2.0**-11)


def test_rows_apart_and_workspace():
    """Queries that are a view of a wider tensor, and a workspace of the caller's."""
    c = KINDS[0]
    w = Shared(c)
    x, want, batch = run(w, w.prefix())
    wide = torch.full((len(x), c.n_q * c.d + 64), 5.0, dtype=torch.float16, device="cuda")
    q = wide[:, 32:32 + c.n_q * c.d].view(len(x), c.n_q, c.d)
    q.copy_(to_dev(x))
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(0xFF)          # NaN, if it were read
    got = w.cache.attend(q, batch, prefix=w.prefix(), workspace=ws)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert w.cache.attend(q[:0], batch, prefix=w.prefix()).shape == (0, c.n_q, c.d)
    for bad in (dict(window=5), dict(workspace=ws[:100]), dict(workspace=ws.cpu()), dict(scale=0.0), dict(prefix=3)):
        with pytest.raises(W4A16Error):
            w.cache.attend(q, batch, **{**dict(prefix=w.prefix()), **bad})


def test_captured_steps_and_changed_groups():
    """One captured call replayed while lengths, groups and shared pages change, other work between the replays; and two
    graphs with workspaces of their own on two streams."""
    c = KINDS[0]
    w = Shared(c)
    w.rng = np.random.default_rng(3)
    x = w.values(sum(w.new), c.n_q)
    q, batch, prefix = to_dev(x), w.batch(w.new, ctx=w.held()), w.prefix()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w.cache.attend(q, batch, prefix=prefix)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.cache.attend(q, batch, prefix=prefix))
        graphs.append(g)
    for step, (cu, pages) in enumerate((([0, 6, 10, 11], [5, 3, 2]), ([0, 6, 6, 6], [4, 1, 1]), ([2, 6, 10, 11], [5, 2, 1]),
                                        ([0, 0, 0, 0], [1, 1, 1]))):
        prefix.cu_seqs.copy_(i32(cu))
        prefix.pages.copy_(i32(pages))
        want = w.cache.attend(q, batch, prefix=w.prefix(pages=pages, cu=cu, max_pages=5))
        torch.randn(1000, device="cuda").sum().item()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o.view(torch.int16), want.view(torch.int16)), step
        w.check(x, want)


@pytest.mark.parametrize("c", [Case(128, 64, 8, 64, ((5, 20),), 150, 1, 0), Case(128, 64, 8, 8, ((5, 3), (3, 2)), 150, 1, 0)])
def test_pages_beyond_4_gib(c):
    """Pools of 4.6 GB for K and for V, pages all over them."""
    w = Shared(c, pool=70001)
    assert int(w.table.max()) * 64 * 8 * 128 > 1 << 32
    x, out, _ = run(w, w.prefix())
    w.check(x, out, weights=weights(c))


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    rng = np.random.default_rng(70 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]
    d, page = pick(64, 96, 128, 256), pick(64, 128, 256)
    n_kv, group = pick((1, 8), (2, 4), (4, 1), (3, 7), (8, 8), (1, 40))
    groups = tuple((int(rng.integers(0, 1 + 900 // page)), int(rng.integers(1, pick(3, 12, 60)))) for _ in range(pick(1, 1, 2, 4)))
    c = Case(d, page, n_kv, n_kv * group, groups, int(rng.integers(1, pick(60, 400, 1500))), pick(1, 1, 1, 3, 6), pick(0, 0, 3, 50))
    w = Shared(c, seed=seed)
    G = len(groups)
    pages = [int(rng.integers(0, p + 2)) if rng.random() < 0.3 else p for p in w.pages]
    most = pick(max(max(w.pages), 1), max(max(w.pages), 1), 1, max(w.pages) + 3)
    front, back = pick(0, 0, 3), pick(0, 0, 9)
    T, B, cols, _, _ = sizes(c)
    print(seed, c, kv.attention_config(T + front + back, B, cols, c.n_q, c.n_kv, d, page, groups=G, max_pages=most), flush=True)
    x, out, batch = run(w, w.prefix(pages=pages, max_pages=most), front=front, back=back, seed=seed)
    w.check(x, out, front=front)
