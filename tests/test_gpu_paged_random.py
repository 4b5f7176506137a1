"""Random calls of the paged cache within its documented limits against the definition:
ragged batches with sequences that are skipped, pages that are not there, pages that took
in an infinity or NaN, windows with sinks, rows apart, tables of any width."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import to_dev
from test_gpu_paged import World
from w4a16_dequant_gemv_amd import kv

pytestmark = pytest.mark.gpu


def sees(n, total, window, sinks, lo, hi):
    """Which of the last n rows see a token of lo .. hi - 1."""
    i = total - n + np.arange(n)[:, None]
    j = np.arange(lo, hi)[None]
    see = j <= i
    if window:
        see &= (i - j < window) | (j < sinks)
    return see.any(1)


@pytest.mark.parametrize("seed", range(48))
def test_random_calls(seed):
    rng = np.random.default_rng(900 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]
    d, page = pick(64, 96, 128, 256), pick(64, 128, 256)
    n_kv, group = pick((1, 8), (2, 4), (4, 1), (1, 1), (3, 7), (2, 16), (8, 8), (1, 40))
    n_q = n_kv * group
    B = pick(1, 2, 3, 7, 66)
    most = pick(256, 700, 1500) if B < 60 else 256
    per = pick(1, 1, 3, 20, 150) if B < 60 else pick(1, 2, 9)
    w = World(B, n_kv, d, page, seed=seed, most=pick(most, 4096, 30000) if B < 60 else most)
    held = rng.integers(0, most + 1, B).tolist()
    new = [int(min(h, rng.integers(0, per + 1))) for h in held]
    if sum(new) == 0:
        held[0], new[0] = max(held[0], 1), 1
    front, back = pick(0, 0, 3), pick(0, 0, 70)

    # prompts in two calls; in some pages a value of one head that is not finite
    k, v = w.values(sum(held), n_kv), w.values(sum(held), n_kv)
    starts = np.concatenate([[0], np.cumsum(held)])
    spoiled = []
    for b, h in enumerate(held):
        clean = k[starts[b]:starts[b + 1]].copy(), v[starts[b]:starts[b + 1]].copy()
        if h >= page and rng.random() < 0.4:
            p, head = int(rng.integers(h // page)), int(rng.integers(n_kv))
            x = pick(k, v)
            x[starts[b] + p * page + int(rng.integers(page)), head, int(rng.integers(d))] = pick(np.nan, np.inf, -np.inf)
            spoiled.append((b, p, head))
        w.seqs[b].append(*clean)
    first = [int(rng.integers(0, h + 1)) for h in held]
    rest = [h - f for h, f in zip(held, first)]
    for n, at in ((first, [0] * B), (rest, first)):
        rows = np.concatenate([starts[b] + at[b] + np.arange(n[b]) for b in range(B)]).astype(int)
        if len(rows):
            w.cache.append(to_dev(k[rows]), to_dev(v[rows]), w.batch(n, ctx=at))

    # the call: some sequences skipped, some pages not there
    window = pick(0, 0, 1, 30, 400)
    sinks = pick(0, 1, 100) if window else 0
    scale = pick(d ** -0.5, d ** -0.5, 0.01, 2.0)
    ctx, slots, table = [h - n for h, n in zip(held, new)], w.slots.copy(), w.table.copy()
    skip = np.zeros(B, bool)
    hidden = [[] for _ in range(B)]
    for b in range(B):
        r = rng.random()
        if B > 1 and r < 0.08:
            skip[b], ctx[b] = True, -1
        elif B > 1 and r < 0.16:
            skip[b], slots[b] = True, pick(-1, B + 2)
        elif held[b] >= page and r < 0.4:
            p = int(rng.integers(held[b] // page))
            hidden[b].append(p)
            table[b, p] = pick(-1, w.cache.pool_pages, 1 << 30)
    T = sum(new) + front + back
    x = w.values(T, n_q)
    wide = torch.full((T, n_q * d + 64), 5.0, dtype=torch.float16, device="cuda")
    q = wide[:, 32:32 + n_q * d].view(T, n_q, d) if rng.random() < 0.5 else wide[:, :n_q * d].view(T, n_q, d)
    q.copy_(to_dev(x))
    out = torch.full((T, n_q, d), 7.0, dtype=torch.float16, device="cuda")
    w.cache.attend(q, w.batch(new, front, ctx=ctx, table=table, slots=slots), scale=scale, window=window, sinks=sinks, out=out)
    torch.cuda.synchronize()
    name = kv.attention_config(T, B, w.cols, n_q, n_kv, d, page, window, sinks)
    print(seed, name, flush=True)
    y = out.cpu().numpy().astype(np.float64)
    assert (y[:front] == 7).all() and (y[T - back:] == 7).all()
    weights = {} if "rows_kernel" in name else dict(weights=ref.WEIGHTS_IN_TWO)
    at = front
    for b, (s, n) in enumerate(zip(w.seqs, new)):
        got = y[at:at + n]
        if n and skip[b]:
            assert (got == 7).all(), b
        elif n:
            o, size, top = ref.attend(s, x[at:at + n], scale, window, sinks, hidden[b])
            ok = np.abs(got - o) <= ref.tolerance(o, size, top, len(s), d, **weights)
            for sb, p, head in spoiled:
                if sb == b and p not in hidden[b]:
                    bad = sees(n, len(s), window, sinks, p * page, (p + 1) * page)
                    heads = slice(head * group, (head + 1) * group)
                    assert np.isnan(got[bad, heads]).all(), (b, p, head)
                    ok[bad, heads] = True
            assert bool(ok.all()), (b, np.argwhere(~ok)[:3].tolist())
        at += n
