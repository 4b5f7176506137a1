"""Attention with shared pages: its refusals, through the C ABI (every call carries an invalid
argument, so nothing is launched) and through the Python wrappers, and the kernels that the sizes of a call choose."""
import ctypes
import re

import pytest
import torch

from shared_cases import CASES, sizes
from w4a16_dequant_gemv_amd import _lib, kv
from w4a16_dequant_gemv_amd._lib import Q4_ERR_ALIGN, Q4_ERR_NULL, Q4_ERR_SHAPE, W4A16Error

P = 0x10000


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def attend(L, cache=None, batch=None, prefix=None, **kw):
    c = _lib.PagedCache(**{**dict(k=P, v=P, k_scale=P, v_scale=P, k_tail=P, v_tail=P, pages=10, slots=4, n_kv=8, d=128,
                                  page=128), **(cache or {})})
    b = _lib.PagedBatch(**{**dict(cu_q=P, ctx_lens=P, block_table=P, slots=P, tokens=3, batch=2, table_cols=5), **(batch or {})})
    p = _lib.SharedPrefix(**{**dict(cu_seqs=P, pages=P, groups=1, max_pages=3), **(prefix or {})})
    a = dict(q=P, qs=8192, n_q=64, scale=0.1, ws=P, size=1 << 40, out=P)
    a.update(kw)
    return L.kv_paged_attention_shared(c, b, p, a["q"], a["qs"], a["n_q"], a["scale"], a["ws"], a["size"], a["out"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(cache=dict(k=None)), Q4_ERR_NULL), (dict(cache=dict(d=80)), Q4_ERR_SHAPE), (dict(cache=dict(page=32)), Q4_ERR_SHAPE),
    (dict(cache=dict(k_tail=P + 2)), Q4_ERR_ALIGN), (dict(batch=dict(cu_q=None)), Q4_ERR_NULL),
    (dict(batch=dict(tokens=0)), Q4_ERR_SHAPE), (dict(batch=dict(batch=65537)), Q4_ERR_SHAPE),
    (dict(batch=dict(table_cols=1 << 24)), Q4_ERR_SHAPE), (dict(batch=dict(slots=P + 1)), Q4_ERR_ALIGN),
    (dict(prefix=dict(cu_seqs=None)), Q4_ERR_NULL), (dict(prefix=dict(pages=None)), Q4_ERR_NULL),
    (dict(prefix=dict(groups=0)), Q4_ERR_SHAPE), (dict(prefix=dict(groups=-1)), Q4_ERR_SHAPE),
    (dict(prefix=dict(groups=65537)), Q4_ERR_SHAPE), (dict(prefix=dict(max_pages=0)), Q4_ERR_SHAPE),
    (dict(prefix=dict(max_pages=(1 << 24) + 1)), Q4_ERR_SHAPE), (dict(prefix=dict(cu_seqs=P + 2)), Q4_ERR_ALIGN),
    (dict(prefix=dict(pages=P + 1)), Q4_ERR_ALIGN), (dict(cache=dict(n_kv=64), prefix=dict(groups=65536)), Q4_ERR_SHAPE),
    (dict(q=None), Q4_ERR_NULL), (dict(ws=None), Q4_ERR_NULL), (dict(out=None), Q4_ERR_NULL), (dict(n_q=60), Q4_ERR_SHAPE),
    (dict(scale=0.0), Q4_ERR_SHAPE), (dict(scale=float("nan")), Q4_ERR_SHAPE), (dict(qs=8184), Q4_ERR_SHAPE),
    (dict(qs=8196), Q4_ERR_SHAPE), (dict(q=P + 8), Q4_ERR_ALIGN), (dict(ws=P + 8), Q4_ERR_ALIGN), (dict(out=P + 2), Q4_ERR_ALIGN),
    (dict(size=1000), Q4_ERR_SHAPE), (dict(size=-1), Q4_ERR_SHAPE)])
def test_refusals(L, bad, code):
    assert attend(L, **bad) == code


def test_null_structs(L):
    c = _lib.PagedCache(k=P, v=P, k_scale=P, v_scale=P, k_tail=P, v_tail=P, pages=10, slots=4, n_kv=8, d=128, page=128)
    b = _lib.PagedBatch(cu_q=P, ctx_lens=P, block_table=P, slots=P, tokens=3, batch=2, table_cols=5)
    null = ctypes.POINTER(_lib.SharedPrefix)()
    assert L.kv_paged_attention_shared(c, b, null, P, 8192, 64, 0.1, P, 1 << 40, P, None) == Q4_ERR_NULL


SIZES = dict(tokens=64, batch=64, table_cols=40, page=128, groups=1, max_pages=32, n_q=64, n_kv=8, d=128)


def size(L, **kw):
    return L.kv_paged_attention_shared_workspace_size(*{**SIZES, **kw}.values())


def test_workspace_size(L):
    for bad in (dict(tokens=0), dict(batch=0), dict(batch=65537), dict(table_cols=0), dict(page=100), dict(groups=0),
                dict(max_pages=0), dict(n_q=60), dict(d=80), dict(table_cols=1 << 24)):
        assert size(L, **bad) == 0, bad
    whole = dict(batch=dict(tokens=64, batch=64, table_cols=40), prefix=dict(groups=1, max_pages=32))
    assert attend(L, **whole, size=size(L) - 1) == Q4_ERR_SHAPE
    assert size(L) >= 64 * 64 * 2 * 130 * 4                    # two parts of a row at least
    # a chunk of a prompt is run as without shared pages, and needs what that needs
    assert size(L, tokens=4096, batch=4) == L.kv_paged_attention_workspace_size(4096, 4, 64, 8, 128)


def name_of(*args, **kw):
    return re.sub(r"\d+ cuts, |\d+ chunks", "", kv.attention_config(*args, **kw))


def case_name(c):
    T, B, cols, G, most = sizes(c)
    return kv.attention_config(T, B, cols, c.n_q, c.n_kv, c.d, c.page, groups=G, max_pages=most)


def test_every_way_has_a_case():
    """The sizes of calls reach every kernel that is built, and the cases reach each of them, with one and with
    several chunks of own tokens."""
    reachable = set()
    for d in (64, 96, 128, 256):
        for n_q, n_kv in ((8, 8), (64, 8), (16, 8), (32, 1), (28, 4)):
            for B in (1, 3, 16, 64, 256, 2000):
                for new in (1, 5):
                    for pages in (1, 8, 64, 1000):
                        for more in (1, 6, 20, 400):
                            if B * new * n_q * d <= 1 << 34:
                                reachable.add(name_of(B * new, B, pages + more, n_q, n_kv, d, 64, groups=1, max_pages=pages))
    want = set()
    for d in (64, 96, 128, 256):
        for many in ("false", "true"):
            for waves in (1, 2, 4):
                if d == 256 and many == "true":
                    want.add(f"kv_shared_rows_kernel<256, 8, 1>, kv_shared_kernel<256, false, 1>, kv_shared_join_kernel<256>, {waves} waves, ")
                else:
                    want.add(f"kv_shared_kernel<{d}, {many}, {2 if d < 256 else 1}>, kv_shared_join_kernel<{d}>, {waves} waves, ")
    assert {n for n in reachable if "kv_attend" not in n} == want
    names = [case_name(c) for c in CASES]
    covered = {re.sub(r"\d+ cuts, |\d+ chunks", "", n) for n in names}
    assert want <= covered, sorted(want - covered)
    assert any(n.endswith(", 1 chunks") for n in names) and any(re.search(r" [2-8] chunks$", n) for n in names)
    assert "kv_attend" in kv.attention_config(4096, 4, 40, 64, 8, 128, groups=1, max_pages=32)


def test_the_report_validates_like_the_entry_point(L):
    buf = ctypes.create_string_buffer(64)
    args = lambda **kw: [*{**SIZES, **kw}.values()]
    f = L.kv_paged_attention_shared_config
    assert f(*args(), buf, 64) == 0 and buf.value.startswith(b"kv_shared_kernel<128, ") and len(buf.value) == 63
    assert f(*args(), None, 64) == Q4_ERR_NULL
    assert f(*args(), buf, 0) == Q4_ERR_SHAPE
    for bad in (dict(tokens=0), dict(batch=0), dict(table_cols=0), dict(page=32), dict(groups=0), dict(max_pages=0),
                dict(n_q=60), dict(d=80)):
        assert f(*args(**bad), buf, 64) == Q4_ERR_SHAPE, bad
    with pytest.raises(W4A16Error):
        kv.attention_config(64, 64, 40, 64, 8, 128, window=10, groups=1, max_pages=32)


def test_python_refuses_cpu_tensors():
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    for args in ((i(0, 2), i(3), 3), (i(0, 2), 3, 3), (i(0), i(), 3), (i(0, 2), i(3).float(), 3)):
        with pytest.raises(W4A16Error):
            kv.SharedPrefix(*args)
