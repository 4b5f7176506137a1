"""Launches of attention over shared pages stay below 2^32 threads for every size that the entry point takes."""
import re

import pytest

from w4a16_dequant_gemv_amd import kv


@pytest.mark.parametrize("tokens,batch,groups,n_q,n_kv,d,cols,pages", [
    (65536 * 8, 65536, 1, 64, 32, 64, 4096, 4), (65536 * 31, 65536, 1, 64, 32, 64, 8192, 100), (65536 * 8, 65536, 65536, 64, 32, 128, 4096, 4),
    (65536 * 60, 65536, 3, 32, 32, 64, 2000, 1), (2048 * 4, 2048, 7, 1024, 1024, 64, 4096, 60), (65536, 65536, 1, 64, 8, 128, 4096, 32),
    (65536 * 15, 65536, 1, 64, 16, 256, 4096, 32), (1, 1, 1, 64, 8, 128, 1 << 16, 1)])
def test_threads(tokens, batch, groups, n_q, n_kv, d, cols, pages):
    page, group = 64, n_q // n_kv
    assert batch * n_kv <= 1 << 21 and groups * n_kv <= 1 << 21 and tokens * n_q * d <= 1 << 34
    name = kv.attention_config(tokens, batch, cols, n_q, n_kv, d, page, groups=groups, max_pages=pages)
    assert "kv_shared" in name
    cuts, waves, chunks = (int(x) for x in re.search(r"(\d+) cuts, (\d+) waves, (\d+) chunks", name).groups())
    rows = 128 if "true" in name or "rows_kernel" in name else 16
    shared = (max(tokens * group - groups, 0) // rows + groups) * n_kv * cuts
    own = -(-(tokens * group // 16 + batch) * n_kv // (4 // waves)) * chunks
    assert (own if "rows_kernel" in name else shared + own) * 256 < 1 << 32, name
    assert shared * (512 if "rows_kernel" in name else 256) < 1 << 32, name
