"""Sequences of the paged cache that go back and on again, over and over, within what
kv_codec.h allows: to the page before the highest one reached, or to a page's border."""
import numpy as np
import pytest

import paged_ref as ref
from gpu_util import to_dev
from test_gpu_paged import World

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,page,n_q,steps,seed", [(64, 64, 4, 60, 0), (128, 128, 2, 40, 1), (96, 256, 8, 30, 2),
                                                   (256, 64, 2, 40, 3)])
def test_back_and_on_within_the_limits(d, page, n_q, steps, seed):
    w = World(3, 2, d, page, seed=seed, most=8 * page)
    rng = np.random.default_rng(seed)
    limit = 8 * page
    highest, border = [0] * 3, [0] * 3                   # the highest page reached, and the last border gone back to
    for step in range(steps):
        for b, s in enumerate(w.seqs):
            low = max((highest[b] - 1) * page, border[b], 0)
            to = len(s)
            if rng.random() < 0.15 or len(s) > limit - page:
                to = page * int(rng.integers(0, len(s) // page + 1))
                if to < low:                             # a border further back: begins anew there
                    highest[b], border[b] = to // page, to
            elif rng.random() < 0.6:
                to = int(rng.integers(low, len(s) + 1))
            s.k, s.v = s.k[:to], s.v[:to]
        n = [int(rng.integers(0, m)) for m in rng.choice([2, 9, page, 2 * page], 3)]
        n = [min(m, limit - len(s)) for m, s in zip(n, w.seqs)]
        if sum(n):
            w.append(n)
            w.attend(n, n_q)
        for b, s in enumerate(w.seqs):
            highest[b] = max(highest[b], (len(s) - 1) // page if len(s) else 0)
        q = w.values(3, n_q)
        got = w.cache.attend(to_dev(q), w.batch([min(len(s), 1) for s in w.seqs],
                                                ctx=[max(len(s) - 1, 0) for s in w.seqs])).cpu().numpy()
        row = 0
        for s in w.seqs:
            if len(s):
                o, size, most = ref.attend(s, q[row:row + 1], d ** -0.5)
                ok = np.abs(got[row].astype(np.float64) - o[0]) <= ref.tolerance(o, size, most, len(s), d)[0]
                assert bool(ok.all()), step
                row += 1
    w.check_storage(ring=False)
