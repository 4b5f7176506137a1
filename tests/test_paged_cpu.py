"""The paged cache's refusals, through the C ABI (every call carries an invalid
argument, so nothing is launched) and through the Python wrappers, and its
definition in `paged_ref` against brute force."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from w4a16_dequant_gemv_amd import _lib, kv
from w4a16_dequant_gemv_amd._lib import Q4_ERR_ALIGN, Q4_ERR_NULL, Q4_ERR_SHAPE, W4A16Error

P = 0x10000


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, k_tail=P, v_tail=P, pages=10, slots=4, n_kv=8, d=128, page=128)
    a.update(kw)
    return _lib.PagedCache(**a)


def batch(**kw):
    a = dict(cu_q=P, ctx_lens=P, block_table=P, slots=P, tokens=3, batch=2, table_cols=5)
    a.update(kw)
    return _lib.PagedBatch(**a)


def append(L, c=None, b=None, **kw):
    a = dict(k=P, ks=1024, v=P, vs=1024, q=P, qs=8192, n_q=64, rope=P, rows=100, dim=128, inter=0, pos=P, out=P)
    a.update(kw)
    return L.kv_paged_append(cache() if c is None else c, batch() if b is None else b, a["k"], a["ks"], a["v"], a["vs"],
                             a["q"], a["qs"], a["n_q"], a["rope"], a["rows"], a["dim"], a["inter"], a["pos"], a["out"],
                             None)


def attend(L, c=None, b=None, **kw):
    a = dict(q=P, qs=8192, n_q=64, scale=0.1, window=0, sinks=0, ws=P, size=1 << 40, out=P)
    a.update(kw)
    return L.kv_paged_attention(cache() if c is None else c, batch() if b is None else b, a["q"], a["qs"], a["n_q"],
                                a["scale"], a["window"], a["sinks"], a["ws"], a["size"], a["out"], None)


BAD_CACHE = [(dict([(n, None)]), Q4_ERR_NULL) for n in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")] + [
    (dict(n_kv=0), Q4_ERR_SHAPE), (dict(n_kv=1025), Q4_ERR_SHAPE), (dict(d=80), Q4_ERR_SHAPE), (dict(d=512), Q4_ERR_SHAPE),
    (dict(page=32), Q4_ERR_SHAPE), (dict(page=512), Q4_ERR_SHAPE), (dict(page=100), Q4_ERR_SHAPE),
    (dict(pages=0), Q4_ERR_SHAPE), (dict(pages=1 << 30), Q4_ERR_SHAPE), (dict(slots=0), Q4_ERR_SHAPE),
    (dict(slots=1 << 24), Q4_ERR_SHAPE), (dict(k=P + 8), Q4_ERR_ALIGN), (dict(v_tail=P + 2), Q4_ERR_ALIGN),
    (dict(k_scale=P + 2), Q4_ERR_ALIGN)]
BAD_BATCH = [(dict([(n, None)]), Q4_ERR_NULL) for n in ("cu_q", "ctx_lens", "block_table", "slots")] + [
    (dict(tokens=0), Q4_ERR_SHAPE), (dict(tokens=-1), Q4_ERR_SHAPE), (dict(tokens=1 << 25), Q4_ERR_SHAPE),
    (dict(batch=0), Q4_ERR_SHAPE), (dict(batch=65537), Q4_ERR_SHAPE), (dict(table_cols=0), Q4_ERR_SHAPE),
    (dict(table_cols=1 << 24), Q4_ERR_SHAPE), (dict(cu_q=P + 2), Q4_ERR_ALIGN), (dict(slots=P + 1), Q4_ERR_ALIGN)]


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_batch_are_checked(L, call):
    null = ctypes.POINTER(_lib.PagedCache)()
    assert call(L, c=null) == Q4_ERR_NULL
    assert call(L, b=ctypes.POINTER(_lib.PagedBatch)()) == Q4_ERR_NULL
    for bad, code in BAD_CACHE:
        assert call(L, c=cache(**bad)) == code, bad
    for bad, code in BAD_BATCH:
        assert call(L, b=batch(**bad)) == code, bad
    assert call(L, c=cache(n_kv=64), b=batch(batch=32769)) == Q4_ERR_SHAPE


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), Q4_ERR_NULL), (dict(v=None), Q4_ERR_NULL), (dict(pos=None), Q4_ERR_NULL), (dict(out=None), Q4_ERR_NULL),
    (dict(ks=1016), Q4_ERR_SHAPE), (dict(vs=1028), Q4_ERR_SHAPE), (dict(qs=8184), Q4_ERR_SHAPE),
    (dict(ks=1 << 34), Q4_ERR_SHAPE), (dict(n_q=60), Q4_ERR_SHAPE), (dict(n_q=0), Q4_ERR_SHAPE), (dict(n_q=2048), Q4_ERR_SHAPE),
    (dict(dim=16), Q4_ERR_SHAPE), (dict(dim=160), Q4_ERR_SHAPE), (dict(dim=48), Q4_ERR_SHAPE), (dict(rows=0), Q4_ERR_SHAPE),
    (dict(k=P + 8), Q4_ERR_ALIGN), (dict(v=P + 2), Q4_ERR_ALIGN), (dict(q=P + 4), Q4_ERR_ALIGN), (dict(out=P + 8), Q4_ERR_ALIGN),
    (dict(rope=P + 8), Q4_ERR_ALIGN), (dict(pos=P + 2), Q4_ERR_ALIGN)])
def test_append_rejects(L, bad, code):
    assert append(L, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), Q4_ERR_NULL), (dict(ws=None), Q4_ERR_NULL), (dict(out=None), Q4_ERR_NULL),
    (dict(n_q=12), Q4_ERR_SHAPE), (dict(qs=100), Q4_ERR_SHAPE), (dict(scale=0.0), Q4_ERR_SHAPE),
    (dict(scale=-1.0), Q4_ERR_SHAPE), (dict(scale=float("nan")), Q4_ERR_SHAPE), (dict(scale=float("inf")), Q4_ERR_SHAPE),
    (dict(window=-1), Q4_ERR_SHAPE), (dict(sinks=-1, window=4), Q4_ERR_SHAPE), (dict(sinks=4), Q4_ERR_SHAPE),
    (dict(size=0), Q4_ERR_SHAPE), (dict(q=P + 8), Q4_ERR_ALIGN), (dict(ws=P + 8), Q4_ERR_ALIGN), (dict(out=P + 2), Q4_ERR_ALIGN)])
def test_attention_rejects(L, bad, code):
    assert attend(L, **bad) == code


def test_workspace_stays_small(L):
    """Parts of rows, not of all rows times sixteen: at most 2^18 of d + 2 floats."""
    for T in (1, 17, 512, 1500, 2800, 5000, 20001, 100000, 1 << 20):
        for B in (1, 2, 4, 64, 512):
            for n_q, n_kv, d in ((8, 1, 256), (32, 32, 128), (64, 8, 128), (64, 8, 64), (24, 8, 96)):
                size = L.kv_paged_attention_workspace_size(T, B, n_q, n_kv, d)
                assert 0 < size <= (1 << 18) * (d + 2) * 4 + (1 << 20), (T, B, n_q, n_kv, d, size)


def test_attention_needs_its_whole_workspace(L):
    for T, B, n_q, n_kv, d in ((3, 2, 64, 8, 128), (1, 1, 1, 1, 64), (5000, 3, 16, 8, 256), (300, 300, 8, 1, 96)):
        size = L.kv_paged_attention_workspace_size(T, B, n_q, n_kv, d)
        assert size > 0
        assert attend(L, c=cache(n_kv=n_kv, d=d), b=batch(tokens=T, batch=B), n_q=n_q, qs=n_q * d, size=size - 1) == Q4_ERR_SHAPE
    for bad in ((0, 2, 64, 8, 128), (3, 0, 64, 8, 128), (3, 2, 60, 8, 128), (3, 2, 64, 8, 100)):
        assert L.kv_paged_attention_workspace_size(*bad) == 0


def test_read_rejects(L):
    def read(c=None, ids=P, n=3, k=P, v=P):
        return L.kv_paged_read(c or cache(), ids, n, k, v, None)
    assert read(ids=None) == Q4_ERR_NULL and read(k=None) == Q4_ERR_NULL and read(v=None) == Q4_ERR_NULL
    assert read(n=0) == Q4_ERR_SHAPE and read(n=1 << 22) == Q4_ERR_SHAPE
    assert read(ids=P + 2) == Q4_ERR_ALIGN and read(k=P + 8) == Q4_ERR_ALIGN
    for bad, code in BAD_CACHE:
        assert read(cache(**bad)) == code


def test_python_refuses_cpu_tensors_and_bad_sizes():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(W4A16Error):
        kv.PagedBatch(i, i[:2], i[:2].view(2, 1), i[:2])
    with pytest.raises(W4A16Error):
        kv.PagedBatch(None, None, None, None)
    for a in ((4, 2, 80, 2), (0, 2, 128, 2), (4, 0, 128, 2), (4, 2, 128, 0)):
        with pytest.raises(W4A16Error):
            kv.PagedKVCache(*a, "cpu")
    with pytest.raises(W4A16Error):
        kv.PagedKVCache(4, 2, 128, 2, "cpu", page=32)
    c = kv.PagedKVCache(4, 2, 128, 2, "cpu")
    with pytest.raises(W4A16Error):
        c.append(torch.zeros(1, 2, 128).half(), torch.zeros(1, 2, 128).half(), None)
    with pytest.raises(W4A16Error):
        c.attend(torch.zeros(1, 2, 128).half(), None)
    with pytest.raises(W4A16Error):
        c.read(i)


def test_rope_table_is_the_references():
    """Cosines by another library's binary64 function may differ by a unit of
    binary64, which moves a binary32 value by at most one unit (2^-24 of 1)."""
    a, b = kv.rope_table(3000, 64, 500000.0, "cpu").numpy(), ref.rope_table(3000, 64, 500000.0)
    assert a.dtype == np.float32 and a.shape == b.shape
    assert np.abs(a.astype(np.float64) - b).max() <= 2.0**-24


# the reference itself

@pytest.mark.parametrize("t,d", [(64, 64), (128, 96), (256, 128)])
def test_page_order_places_every_value_once(t, d):
    x = np.arange(t * d).reshape(t, d)
    k, v = ref.page_order(x, "k"), ref.page_order(x, "v")
    assert np.array_equal(np.sort(k), x.ravel()) and np.array_equal(np.sort(v), x.ravel())
    kk = k.reshape(t // 64, 4, d // 16, 16, 16)
    vv = v.reshape(t // 16, d, 16)
    for i, m, a, c, e in ((0, 0, 0, 0, 0), (0, 5, 2, 1, 7), (t // 64 - 1, 15, 3, d // 16 - 1, 15)):
        assert kk[i, a, c, m, e] == x[64 * i + 16 * (m // 4) + 4 * a + m % 4, 16 * c + e]
    assert vv[1, 5, 3] == x[19, 5]


def test_reference_attention_by_brute_force():
    rng = np.random.default_rng(0)
    s = ref.Sequence(1, 64, 64)
    s.append(*(rng.standard_normal((100, 1, 64)).astype(np.float16) for _ in range(2)))
    q = rng.standard_normal((3, 2, 64)).astype(np.float16)
    o, _, _ = ref.attend(s, q, 0.2, window=5, sinks=2)
    for i in range(3):
        at = 97 + i
        js = [j for j in range(at + 1) if at - j < 5 or j < 2]
        for h in range(2):
            w, acc = 0.0, np.zeros(64)
            for j in js:
                k, v = s.k[j, 0].astype(float), s.v[j, 0].astype(float)
                if j < 64:
                    (ck, sk), (cv, sv) = ref.quantize(s.k[:64, 0]), ref.quantize(s.v[:64, 0])
                    k, v = ck[j].astype(float) * float(sk), cv[j].astype(float) * float(sv)
                p = np.exp(0.2 * float(q[i, h].astype(float) @ k))
                w, acc = w + p, acc + p * v
            assert np.allclose(o[i, h], acc / w, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("mistake", ["causal", "window", "sinks", "scale", "tail", "order"])
def test_reference_notices_planted_mistakes(mistake):
    """The tolerance is small enough to see each of these in the oracle."""
    rng = np.random.default_rng(1)
    s = ref.Sequence(1, 64, 64)
    s.append(*(rng.standard_normal((150, 1, 64)).astype(np.float16) for _ in range(2)))
    q = rng.standard_normal((2, 1, 64)).astype(np.float16)
    o, size, most = ref.attend(s, q, 0.125, window=40, sinks=3)
    tol = ref.tolerance(o, size, most, 150, 64)
    if mistake == "causal":
        bad = ref.attend(s, np.concatenate([q, q])[1:3], 0.125, 40, 3)[0][::-1]
    elif mistake == "window":
        bad = ref.attend(s, q, 0.125, 41, 3)[0]
    elif mistake == "sinks":
        bad = ref.attend(s, q, 0.125, 40, 2)[0]
    elif mistake == "scale":
        bad = ref.attend(s, q, 0.124, 40, 3)[0]
    elif mistake == "tail":
        t = ref.Sequence(1, 64, 64)
        t.append(s.k.copy(), np.concatenate([s.v[:149], s.v[148:149]]))
        bad = ref.attend(t, q, 0.125, 40, 3)[0]
    else:
        t = ref.Sequence(1, 64, 64)
        t.append(s.k, s.v[:, :, ::-1])
        bad = ref.attend(t, q, 0.125, 40, 3)[0]
    assert (np.abs(bad - o) > tol).any()
