"""What a test of the weights' exactness can see: rounding them to one fp16 part, planted in
the definition, is outside the tolerance for two parts and inside that for one."""
import numpy as np
import pytest

import paged_ref as ref


@pytest.mark.parametrize("d,page,tokens", [(64, 64, 330), (128, 128, 330), (96, 64, 200), (256, 64, 200), (96, 128, 300)])
def test_one_part_is_seen(d, page, tokens):
    n_kv = 8
    k, v, q, scale = ref.balanced(n_kv, d, tokens)
    s = ref.Sequence(n_kv, d, page)
    s.append(k, v)
    o, size, top = ref.attend(s, q, scale)
    got = np.zeros_like(o)
    for h in range(n_kv):
        kh, vh, _ = s.values(h)
        e = scale * (kh @ q[0, h].astype(np.float64))
        p = np.exp(e - e.max()) * 2.0**10
        got[0, h] = p.astype(np.float16).astype(np.float64) @ vh / p.sum()
    err = np.abs(got - o)
    assert (err > ref.tolerance(o, size, top, tokens, 0, ref.WEIGHTS_IN_TWO)).any(-1).sum() >= 2
    assert (err <= ref.tolerance(o, size, top, tokens, d)).all()
