"""The attention's cases run every kernel that the sizes of a call can choose.  Runs on the
CPU: the library's selection report makes no HIP call."""
import ctypes
import re

import pytest

from paged_cases import CASES, Case, table_cols, tokens
from w4a16_dequant_gemv_amd import W4A16Error, kv
from w4a16_dequant_gemv_amd._lib import Q4_ERR_NULL, Q4_ERR_SHAPE, lib

# Sizes around the rules' thresholds: rows of 16, 32, 48 and more a sequence and kv head, one to
# many row blocks on the card's CUs, tables of one page to thousands.
HEADS = ((1, 1), (2, 1), (8, 1), (32, 1), (64, 1), (1024, 1), (8, 8), (64, 8), (32, 32), (64, 16), (64, 64), (1024, 1024),
         (21, 3))
BATCH = (1, 2, 4, 8, 16, 33, 64, 128, 256, 1024, 4096, 65536)
NEW = (1, 2, 3, 5, 6, 8, 12, 17, 24, 40, 48, 49, 64, 100, 128, 200, 257, 400, 700, 1000, 1100, 2100, 5000, 20000)
COLS = (1, 2, 4, 8, 16, 32, 64, 256, 2048)


def name_of(*args, **kw):
    return re.sub(r", \d+ cuts", "", kv.attention_config(*args, **kw))


@pytest.fixture(scope="module")
def reachable():
    out = {}
    for d in (64, 96, 128, 256):
        for n_q, n_kv in HEADS:
            for B in BATCH:
                for new in NEW:
                    if B * n_kv > 1 << 21 or B * new > 1 << 22:
                        continue
                    for cols in COLS:
                        for window in (0, 100):
                            args = (B * new, B, cols, n_q, n_kv, d, 64, window)
                            try:
                                out.setdefault(name_of(*args), args)
                            except W4A16Error:
                                assert B * new * n_q * d > 1 << 34
    return out


@pytest.fixture(scope="module")
def covered():
    return {name_of(tokens(c), c.batch, table_cols(c), c.n_q, c.n_kv, c.d, c.page, c.window): c for c in CASES}


def test_every_way_has_a_case(reachable, covered):
    missing = {n: a for n, a in reachable.items() if n not in covered}
    assert not missing, f"add to tests/paged_cases.py: {missing}"
    assert not [c for n, c in covered.items() if n not in reachable]


def test_every_kernel_in_the_library_is_reached(reachable):
    """Nothing is built that no call reaches: each kernel's sizes as its launch code has them."""
    want = set()
    for d in (64, 96, 128, 256):
        for qt in (1,) if d == 256 else (1, 2, 3):
            occ = 2 if (d <= 64 and qt <= 2) or (d <= 128 and qt == 1) else 1
            split = f"kv_attend_split_kernel<{d}, {qt}, {occ}>"
            want |= {f"{split}, kv_join_kernel<{d}, {qt}, {nw}>" for nw in (1, 4)}
            want |= {f"{split}, whole row blocks", f"kv_attend_wave_kernel<{d}, {qt}, {occ}>"}
        for nw in (8,) if d == 256 else (4, 8):
            rows = f"kv_attend_rows_kernel<{d}, {nw}, {1 if d == 256 else 2}>"
            want |= {rows, f"{rows}, kv_join_rows_kernel<{d}>"}
    assert set(reachable) == want


def test_a_wide_table_or_many_rows_choose_otherwise():
    """The rules' sides that the documents give figures for."""
    one = dict(n_q=32, n_kv=32, d=128, page=128)
    assert "whole" in kv.attention_config(1, 1, 5, **one)
    assert "join" in kv.attention_config(1, 1, 40, **one)
    layout = dict(n_q=64, n_kv=8, d=128, page=128)
    assert "wave" in kv.attention_config(256, 256, 3, **layout)
    assert "split_kernel<128, 1, 2>, kv_join_kernel<128, 1, 1>" in kv.attention_config(256, 256, 32, **layout)
    assert "split_kernel<128, 3, 1>, kv_join" in kv.attention_config(40, 8, 33, **layout)      # five drafted tokens
    assert kv.attention_config(2048, 1, 65, **layout) == "kv_attend_rows_kernel<128, 8, 2>"


def test_the_report_validates_like_the_entry_point():
    L, name = lib(), ctypes.create_string_buffer(100)

    def ask(tokens=3, batch=2, cols=5, page=128, n_q=64, n_kv=8, d=128, window=0, sinks=0, to=name, size=100):
        return L.kv_paged_attention_config(tokens, batch, cols, page, n_q, n_kv, d, window, sinks, to, size)
    assert ask() == 0 and name.value.startswith(b"kv_attend_")
    assert ask(to=None) == Q4_ERR_NULL
    for bad in (dict(tokens=0), dict(tokens=1 << 25), dict(batch=0), dict(batch=65537), dict(cols=0), dict(cols=1 << 24),
                dict(page=100), dict(n_q=60), dict(n_q=0), dict(n_kv=0), dict(d=80), dict(window=-1), dict(sinks=4),
                dict(sinks=-1, window=4), dict(size=0), dict(n_kv=64, batch=32769), dict(tokens=1 << 24, n_q=1024, n_kv=1)):
        assert ask(**bad) == Q4_ERR_SHAPE, bad
    assert ask(size=8) == 0 and len(name.value) == 7
    with pytest.raises(W4A16Error):
        kv.attention_config(1, 1, 1, 3, 2, 64)


def test_cases_are_well_formed():
    assert len(set(CASES)) == len(CASES)
    for c in CASES:
        assert isinstance(c, Case) and c.limit >= c.held >= c.new
