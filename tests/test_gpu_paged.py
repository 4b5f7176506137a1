"""The paged INT8 cache on the GPU against its definition in 64 bits: appended
pages, rings and rotated queries bit for bit, attention within its roundings."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from w4a16_dequant_gemv_amd import kv

pytestmark = pytest.mark.gpu


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy()


class World:
    """A cache on the GPU and the same sequences as the definition has them."""

    def __init__(self, B, n_kv, d, page, pool=None, most=1024, seed=0, dead=True):
        self.rng = np.random.default_rng(seed)
        self.B, self.n_kv, self.d, self.page = B, n_kv, d, page
        self.cols = most // page + 2
        pool = pool or B * self.cols + 2
        self.cache = kv.PagedKVCache(pool, n_kv, d, B + 2, torch.device("cuda"), page=page)
        if dead:                    # what is never written must never matter
            self.cache.k_tail.fill_(float("nan"))
            self.cache.v_tail.fill_(float("nan"))
            self.cache.k.fill_(0x55)
            self.cache.v.fill_(0x55)
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("nan"))
        self.table = self.rng.permutation(pool)[:B * self.cols].reshape(B, self.cols).astype(np.int32)
        self.slots = self.rng.permutation(B + 2)[:B].astype(np.int32)
        self.seqs = [ref.Sequence(n_kv, d, page) for _ in range(B)]

    def batch(self, n, front=0, ctx=None, table=None, slots=None):
        cu = front + np.concatenate([[0], np.cumsum(n)])
        ctx = [len(s) for s in self.seqs] if ctx is None else ctx
        i32 = [np.ascontiguousarray(x, np.int32) for x in (cu, ctx, self.table if table is None else table,
                                                           self.slots if slots is None else slots)]
        return kv.PagedBatch(*(to_dev(x) for x in i32))

    def values(self, T, heads, spread=1.0):
        x = self.rng.standard_normal((T, heads, self.d)) * spread
        x[:, :, 3] *= 6
        return x.astype(np.float16)

    def append(self, n, n_q=None, table=None, positions=None, interleaved=False, fused=False, front=0, back=0):
        """New tokens n[b] for every sequence, on both sides; -> GPU q, expected q."""
        T = sum(n) + front + back
        n_q = n_q or self.n_kv
        x = self.values(T, n_q + 2 * self.n_kv)
        q, k, v = x[:, :n_q], x[:, n_q:n_q + self.n_kv], x[:, n_q + self.n_kv:]
        if positions is None:
            positions = np.concatenate([np.full(front, 0)] + [len(s) + np.arange(m) for s, m in zip(self.seqs, n)]
                                       + [np.full(back, 0)]).astype(np.int32)
        if fused:
            g = to_dev(x)
            gq, gk, gv = g[:, :n_q], g[:, n_q:n_q + self.n_kv], g[:, n_q + self.n_kv:]
        else:
            gq, gk, gv = (to_dev(y) for y in (q, k, v))
        b = self.batch(n, front)
        if table is None:
            out = self.cache.append(gk, gv, b)
            rq, rk = None, k
        else:
            out = self.cache.append(gk, gv, b, q=gq, rope=to_dev(table), positions=to_dev(positions),
                                    interleaved=interleaved)
            rq, rk = (ref.rotate(y, table, positions, interleaved) for y in (q, k))
        at = front
        for s, m in zip(self.seqs, n):
            s.append(rk[at:at + m], v[at:at + m])
            at += m
        return out, rq

    def check_storage(self, ring=True):
        """Every full page and the ring's last two pages, bit for bit."""
        torch.cuda.synchronize()
        k, v = (x.cpu().numpy().reshape(x.shape[0], self.n_kv, -1) for x in (self.cache.k, self.cache.v))
        ks, vs = (x.cpu().numpy() for x in (self.cache.k_scale, self.cache.v_scale))
        kt, vt = (x.cpu().numpy().reshape(x.shape[0], 2, self.n_kv, -1) for x in (self.cache.k_tail, self.cache.v_tail))
        t = self.page
        for b, s in enumerate(self.seqs):
            L = len(s)
            for p in range(L // t):
                for h in range(self.n_kv):
                    for which, x, pool, scale in (("k", s.k, k, ks), ("v", s.v, v, vs)):
                        c, sc = ref.quantize(x[p * t:(p + 1) * t, h])
                        at = self.table[b, p]
                        assert scale[at, h] == sc, (b, p, h, which, scale[at, h], sc)
                        assert np.array_equal(pool[at, h], ref.page_order(c, which)), (b, p, h, which)
            for p in range(max(0, -(-L // t) - 2), -(-L // t)) if ring else ():
                for which, x, tail in (("k", s.k, kt), ("v", s.v, vt)):
                    for h in range(self.n_kv):
                        y = x[p * t:(p + 1) * t, h]
                        want = np.zeros((t, self.d), np.float16)
                        want[:len(y)] = y
                        there = np.zeros((t, self.d), bool)
                        there[:len(y)] = True
                        there = ref.page_order(there, which)
                        got = tail[self.slots[b], p % 2, h]
                        assert np.array_equal(got[there].view(np.int16),
                                              ref.page_order(want, which)[there].view(np.int16)), (b, p, h, which)

    def attend(self, n, n_q, front=0, back=0, spread=1.0, hidden=(), table=None, check=True, **kw):
        """The last n[b] tokens' queries against the definition; -> (q, out)."""
        T = sum(n) + front + back
        x = self.values(T, n_q, spread)
        out = torch.full((T, n_q, self.d), 7.0, dtype=torch.float16, device="cuda")
        b = self.batch(n, front, ctx=[len(s) - m for s, m in zip(self.seqs, n)], table=table)
        got = self.cache.attend(to_dev(x), b, out=out, **kw)
        torch.cuda.synchronize()
        if check:
            self.compare(got, x, n, front, back, hidden, **kw)
        return x, got

    def compare(self, got, x, n, front=0, back=0, hidden=(), scale=None, window=0, sinks=0):
        y = got.cpu().numpy().astype(np.float64)
        assert (y[:front] == 7).all() and (y[len(y) - back:] == 7).all(), "padding rows were written"
        scale = self.d ** -0.5 if scale is None else scale
        at = front
        for i, (s, m) in enumerate(zip(self.seqs, n)):
            if m:
                o, size, most = ref.attend(s, x[at:at + m], scale, window, sinks, hidden)
                tol = ref.tolerance(o, size, most, len(s), self.d)
                err = np.abs(y[at:at + m] - o)
                ok = bool((err <= tol).all())
                assert ok, (i, float((err / tol).max()), np.argwhere(~(err <= tol))[:3].tolist())
            at += m


TABLE = ref.rope_table(2048, 128)


@pytest.mark.parametrize("d,page,n_kv,n_q,steps", [
    (128, 128, 2, 4, [[300, 1, 127], [1, 1, 1], [84, 127, 0], [1, 0, 5]]),
    (64, 64, 1, 1, [[63], [1], [1], [200], [64]]),
    (96, 128, 3, 3, [[128, 129], [255, 1], [1, 126]]),
    (256, 256, 1, 2, [[256, 700], [1, 68], [511, 1]]),
    (128, 64, 2, 16, [[0, 1, 0, 64, 65], [7, 7, 7, 7, 7], [1, 56, 57, 58, 0]]),
    (64, 256, 1, 3, [[1000], [24], [1]]),
    (96, 64, 1, 2, [[5, 64], [123, 64]]),
    (256, 64, 2, 2, [[130], [62], [3]]),
])
@pytest.mark.parametrize("fused", [False, True])
def test_append_bit_exact(d, page, n_kv, n_q, steps, fused):
    w = World(len(steps[0]), n_kv, d, page, seed=d + page)
    table = ref.rope_table(1100, d)
    for n in steps:
        if sum(n):
            got, want = w.append(n, n_q, table, fused=fused)
            assert np.array_equal(bits(got), want.view(np.int16))
            w.check_storage()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dim", [(128, 128), (128, 32), (256, 64), (96, 96), (64, 64), (96, 32)])
def test_rotation_forms(d, dim, interleaved):
    w = World(2, 2, d, 64, seed=dim)
    table = ref.rope_table(5000, dim, base=500000.0)
    T = 150
    pos = w.rng.integers(0, 5000, T).astype(np.int32)          # any positions, any order
    got, want = w.append([100, 50], 6, table, positions=pos, interleaved=interleaved)
    assert np.array_equal(bits(got), want.view(np.int16))
    w.check_storage()


def test_rotation_of_extreme_values():
    """fp16's subnormals, its largest values (a sum beyond them is infinite) and zeros."""
    d, T = 128, 64
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((T, 1, d)) * 10.0 ** rng.uniform(-8, 4.7, (T, 1, d))).clip(-65504, 65504).astype(np.float16)
    x[5] = 0
    x[6] = 65504
    pos = np.arange(T, dtype=np.int32)
    table = ref.rope_table(T, d)
    c = kv.PagedKVCache(1, 1, d, 1, torch.device("cuda"))
    one = [to_dev(np.array(v, np.int32)) for v in ([0, T], [0], [[0]], [0])]
    got = c.append(to_dev(x), to_dev(x), kv.PagedBatch(*one), q=to_dev(x), rope=to_dev(table), positions=to_dev(pos))
    torch.cuda.synchronize()
    assert np.array_equal(bits(got), ref.rotate(x, table, pos).view(np.int16))


def test_rotation_beyond_the_table_is_nan():
    w = World(1, 1, 64, 64, seed=1)
    table = ref.rope_table(10, 64)
    pos = np.array([0, 9, 10, -1, 2147483647, 3], np.int32)
    got, want = w.append([6], 2, table, positions=pos)
    assert np.array_equal(np.isnan(got.cpu().numpy()), np.isnan(want)) and np.isnan(want[2]).all()
    assert np.array_equal(bits(got)[[0, 1, 5]], want.view(np.int16)[[0, 1, 5]])


def test_append_without_rotation_matches_the_codec_map():
    """V's codes and scales are those of the per-token map over a page's values."""
    w = World(1, 1, 64, 64, seed=5)
    w.append([64])
    torch.cuda.synchronize()
    w.check_storage()
    q, s = kv.quant_tokens(to_dev(w.seqs[0].v.reshape(8, 512)))
    assert float(w.cache.v_scale[w.table[0, 0], 0]) == float(s.max())


@pytest.mark.parametrize("parts", [[700], [128, 128, 128, 128, 128, 60], [1] * 30 + [670], [300, 1, 399], [127, 2, 571]])
def test_pages_do_not_depend_on_how_tokens_were_split(parts):
    rng = np.random.default_rng(9)
    k, v = (rng.standard_normal((700, 2, 128)).astype(np.float16) for _ in range(2))
    pos = np.arange(700, dtype=np.int32)
    w = World(1, 2, 128, 128, seed=2)
    at = 0
    for n in parts:
        b = w.batch([n])
        w.cache.append(to_dev(k[at:at + n]), to_dev(v[at:at + n]), b, rope=to_dev(TABLE), positions=to_dev(pos[at:at + n]))
        w.seqs[0].append(ref.rotate(k[at:at + n], TABLE, pos[at:at + n]), v[at:at + n])
        at += n
    w.check_storage()


def test_padding_rows_and_empty_sequences():
    w = World(4, 2, 128, 64, seed=11)
    before = [x.clone() for x in (w.cache.k, w.cache.k_tail)]
    got, want = w.append([0, 70, 0, 3], 4, TABLE, front=5, back=9)
    assert np.array_equal(bits(got), want.view(np.int16))               # q is rotated for every row
    w.check_storage()
    used = [int(w.slots[1]), int(w.slots[3])]
    other = [s for s in range(6) if s not in used]
    assert torch.equal(w.cache.k_tail[other].view(torch.int16), before[1][other].view(torch.int16))
    w.attend([0, 70, 0, 3], 4, front=5, back=9)
    w.attend([0, 1, 0, 1], 4, front=0, back=62)


def test_skipped_sequences_and_pages_write_nothing():
    """Slots, lengths and pages out of range: nothing is stored for them."""
    B, d, page = 6, 64, 64
    w = World(B, 1, d, page, seed=4)
    pool = w.cache.pool_pages
    table = w.table.copy()
    ctx = np.array([0, -1, 0, 0, 0, w.cols * page], np.int32)            # 1: negative, 5: its page is beyond the table
    slots = w.slots.copy()
    slots[2], slots[3] = -1, B + 2
    table[4, 0] = pool                                                   # 4: its full page has nowhere to go
    n = [64, 64, 64, 64, 70, 64]
    x = w.values(sum(n), 1)
    before = [t.clone() for t in (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale, w.cache.k_tail, w.cache.v_tail)]
    b = w.batch(n, ctx=ctx, table=table, slots=slots)
    w.cache.append(to_dev(x), to_dev(x), b)
    torch.cuda.synchronize()
    after = (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale, w.cache.k_tail, w.cache.v_tail)
    for old, new in zip(before[:4], after[:4]):
        same = (old.view(torch.uint8) == new.view(torch.uint8)).flatten(1).all(1)
        assert torch.nonzero(~same).flatten().tolist() == [int(table[0, 0])]
    for old, new in zip(before[4:], after[4:]):
        same = (old.view(torch.int16) == new.view(torch.int16)).flatten(1).all(1)
        assert sorted(torch.nonzero(~same).flatten().tolist()) == sorted([int(slots[0]), int(slots[4])])
    out = torch.full((sum(n), 1, d), 7.0, dtype=torch.float16, device="cuda")
    w.cache.attend(to_dev(x), b, out=out)
    torch.cuda.synchronize()
    y = out.cpu().numpy()
    assert (y[64:256] == 7).all() and (y[326:] == 7).all()               # skipped: their rows stay
    assert np.isfinite(y).all() and not (y[:64] == 7).all()
    # sequence 4: its full page is nowhere, so the rows in it see nothing and give zeros
    assert (y[256:320] == 0).all() and (y[320:326] != 0).any()


def test_read():
    for d, page in ((128, 128), (64, 256), (96, 64), (256, 64)):
        w = World(2, 3, d, page, seed=8)
        w.append([2 * page + 3, page])
        ids = np.array([w.table[0, 1], -1, w.table[1, 0], w.cache.pool_pages, w.table[0, 0]], np.int32)
        ko, vo = (torch.full((5, 3, page, d), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
        w.cache.read(to_dev(ids), ko, vo)
        torch.cuda.synchronize()
        for out, x in ((ko, "k"), (vo, "v")):
            out = out.cpu().numpy()
            assert (out[[1, 3]] == 9).all()
            for i, (b, p) in ((0, (0, 1)), (2, (1, 0)), (4, (0, 0))):
                for h in range(3):
                    c, s = ref.quantize(getattr(w.seqs[b], x)[p * page:(p + 1) * page, h])
                    want = (c.astype(np.float32) * s).astype(np.float16)
                    assert np.array_equal(out[i, h].view(np.int16), want.view(np.int16)), (d, page, x, i, h)


# (d, page, n_kv, n_q, tokens held, queries)
ATTEND = [
    (128, 128, 2, 2, [1], [1]),
    (128, 128, 2, 16, [1, 2, 63, 64, 65, 127, 128, 129, 500], [1] * 9),
    (128, 128, 1, 8, [1000, 3, 640], [1, 3, 2]),
    (64, 64, 3, 12, [64, 200, 130], [1, 1, 1]),
    (64, 64, 2, 8, [400, 17, 256], [5, 5, 5]),
    (96, 128, 2, 14, [300, 129], [2, 1]),
    (256, 256, 1, 4, [700, 256, 255], [1, 1, 1]),
    (256, 64, 2, 4, [300, 64], [20, 1]),
    (128, 64, 1, 32, [333], [4]),
    (128, 128, 1, 64, [260], [1]),
    (64, 128, 1, 71, [200, 130], [1, 2]),
    (128, 256, 2, 8, [800], [300]),
    (128, 128, 1, 1, [700], [700]),
    (96, 64, 2, 2, [190, 64, 1], [190, 64, 1]),
    (256, 64, 1, 2, [200, 333], [77, 130]),
    (64, 64, 1, 8, [900, 100, 64, 500], [129, 0, 64, 1]),
    (128, 128, 2, 4, [0, 300, 0], [0, 40, 0]),
]


@pytest.mark.parametrize("d,page,n_kv,n_q,held,n", ATTEND)
def test_attend(d, page, n_kv, n_q, held, n):
    w = World(len(held), n_kv, d, page, seed=sum(held) + d)
    w.append(held)
    w.attend(n, n_q)
    w.attend(n, n_q, spread=5.0, scale=0.31)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 4), (130, 64), (37, 200), (5000, 4), (300, 100000)])
@pytest.mark.parametrize("d,page,n_kv,n_q,held,n", [
    (128, 128, 2, 16, [1000, 130, 64, 1], [1, 1, 1, 1]),
    (64, 64, 1, 4, [700, 65], [5, 3]),
    (128, 64, 1, 8, [600, 300], [200, 300]),
    (256, 256, 1, 2, [520], [100]),
])
def test_window_and_sinks(d, page, n_kv, n_q, held, n, window, sinks):
    """Pages that no row sees are not in the block table any more."""
    w = World(len(held), n_kv, d, page, seed=window + sinks)
    w.append(held)
    table = w.table.copy()
    for b, (L, m) in enumerate(zip(held, n)):
        for p in range(L // page):
            seen = any(i - j < window or j < sinks for i in (L - m, L - 1) for j in (p * page, (p + 1) * page - 1))
            if not seen and (p + 1) * page <= L - m - window:
                table[b, p] = -1
    w.attend(n, n_q, table=table, window=window, sinks=sinks)


def test_hidden_pages():
    """Pages missing from the block table are not seen; a row without any token gives zeros."""
    w = World(2, 1, 128, 64, seed=21)
    w.append([256, 300])
    table = w.table.copy()
    table[:, 1], table[:, 3] = -5, 10**6
    w.attend([1, 1], 8, table=table, hidden=(1, 3))
    table[:, :] = -1
    _, out = w.attend([200, 200], 8, table=table, hidden=range(9))
    assert (out[:200] == 0).all()


@pytest.mark.parametrize("back", [1, 5, 100, 130])
def test_shortened_sequences(back):
    """Tokens taken back, down to the page before the last one, and others put in their place."""
    w = World(2, 2, 128, 128, seed=back)
    w.append([200, 100])
    w.append([60, 3])
    w.append([130, 160])
    w.append([2, 25])
    for s in w.seqs:
        s.k, s.v = s.k[:len(s) - back], s.v[:len(s) - back]
    w.attend([1, 1], 4)
    w.append([140, 7])
    w.check_storage(ring=False)     # a page before the one it was shortened to may be gone from the ring
    w.attend([1, 3], 4)


@pytest.mark.parametrize("n_q,n,rows", [(8, 1, 6), (32, 40, 2)])
def test_values_that_overflow_nothing(n_q, n, rows):
    """Scores of hundreds, one token that takes all the weight, pages whose
    scales differ by 2^20, zero pages: against the definition."""
    w = World(1, 1, 128, 64, seed=n_q)
    x = w.values(500, 2)
    x[64:128] *= np.float16(2.0**-10)
    x[128:192] = 0
    x[192:256] = np.clip(x[192:256].astype(np.float32) * 1000, -60000, 60000).astype(np.float16)
    x[300, 0] *= 20
    k, v = x[:, :1], x[:, 1:]
    w.cache.append(to_dev(k), to_dev(v), w.batch([500]))
    w.seqs[0].append(k, v)
    w.attend([n], n_q)
    w.attend([n], n_q, scale=1e-4)


def test_infinite_scores_stay_with_their_rows():
    """An infinite query makes its own rows NaN or one-hot and no other's."""
    w = World(2, 1, 64, 64, seed=2)
    w.append([100, 100])
    x = w.values(2, 4)
    x[0, 1] = np.inf
    b = w.batch([1, 1], ctx=[99, 99])
    y = w.cache.attend(to_dev(x), b).cpu().numpy()
    x2 = x.copy()
    x2[0, 1] = 1
    z = w.cache.attend(to_dev(x2), b).cpu().numpy()
    keep = np.ones((2, 4), bool)
    keep[0, 1] = False
    assert np.array_equal(y[keep], z[keep]) and np.isfinite(y[keep]).all()


def test_results_repeat():
    w = World(5, 2, 128, 128, seed=31, most=4096)
    w.append([3000, 17, 900, 2048, 1])
    for n in ([1] * 5, [300, 17, 1, 40, 1]):
        x, a = w.attend(n, 16, check=False)
        for _ in range(3):
            b = w.cache.attend(to_dev(x), w.batch(n, ctx=[len(s) - m for s, m in zip(w.seqs, n)]))
            torch.cuda.synchronize()
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_many_short_sequences():
    rng = np.random.default_rng(6)
    held = rng.integers(1, 200, 150).tolist()
    w = World(150, 1, 64, 64, seed=6, most=256)
    w.append(held, 4, ref.rope_table(256, 64))
    w.check_storage()
    w.attend([1] * 150, 4)
    w.attend([min(3, h) for h in held], 4)


def test_long_context_and_pool_beyond_32_bits():
    """A pool of more than 2^32 bytes: the same pages at its end and at its start
    give the same bits, and the end is right by the definition."""
    d, page, n_kv = 128, 128, 8
    pages = (1 << 32) // (d * page * n_kv) + 40
    w = World(1, n_kv, d, page, pool=64, most=4096, seed=12, dead=False)
    small = w.cache
    w.append([4000])
    x, a = w.attend([1], 32)
    big = kv.PagedKVCache(pages, n_kv, d, 3, torch.device("cuda"), page=page)
    w.cache = big
    w.table = (pages - 1 - np.arange(w.cols, dtype=np.int32))[None].copy()
    s = w.seqs[0]
    w.seqs = [ref.Sequence(n_kv, d, page)]
    w.cache.append(to_dev(s.k), to_dev(s.v), w.batch([4000]))
    w.seqs = [s]
    b = w.cache.attend(to_dev(x), w.batch([1], ctx=[3999]))
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert small is not big
    del big, w.cache
    torch.cuda.empty_cache()
