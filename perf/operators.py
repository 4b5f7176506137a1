"""The paged 8-bit KV cache: appending with rotation, attention over it, and
attention with a sliding window and sinks, as cases that can be timed.

A cache page holds `page` tokens of one sequence, for every kv head, as int8
codes with one fp32 scale per (page, head) for K and one for V.  The last two
pages of a sequence are also kept in fp16 (the ring); a page that is not full
yet is read from there.  Inside a page, K lies as [page/64][4][d/16][16][16]
(token 64*i + 16*(m/4) + 4*a + m%4 of channel 16*c + e at [i][a][c][m][e]) and
V as [page/16][d][16].
"""
import json
import random

import numpy as np
import torch

own = False

# Head layouts: 7B has 32 heads of 128 channels, each with its own K and V;
# 70B has 64 query heads on 8 kv heads.


def listed():
    return [
        # one token of one conversation on the 7B layout; it fills its page
        dict(name="append_7b_1", op="append", batch=1, n_q=32, n_kv=32, d=128, page=128, ctx=639, new=1, ragged=False),
        # a serving step: one token for each of 64 sequences on the 70B layout
        dict(name="append_70b_64", op="append", batch=64, n_q=64, n_kv=8, d=128, page=128, ctx=6000, new=1, ragged=True),
        # prompts of three requests in one call, their ends inside pages
        dict(name="append_prompts", op="append", batch=3, n_q=64, n_kv=8, d=128, page=128, ctx=0, new=5000, ragged=True),
        # one token, one short conversation: latency
        dict(name="decode_7b_1", op="attend", batch=1, n_q=32, n_kv=32, d=128, page=128, ctx=500, new=1, ragged=False,
             window=0, sinks=0),
        # a serving step over ragged contexts up to 4k
        dict(name="decode_70b_64_ragged", op="attend", batch=64, n_q=64, n_kv=8, d=128, page=128, ctx=4096, new=1,
             ragged=True, window=0, sinks=0),
        # the cache that the codec's benchmark quantizes: 32 sequences of 32k tokens
        dict(name="decode_70b_32_32k", op="attend", batch=32, n_q=64, n_kv=8, d=128, page=128, ctx=32767, new=1,
             ragged=False, window=0, sinks=0),
        # one long document
        dict(name="decode_70b_1_128k", op="attend", batch=1, n_q=64, n_kv=8, d=128, page=128, ctx=131000, new=1,
             ragged=False, window=0, sinks=0),
        # five drafted tokens per sequence against their contexts, small heads and pages
        dict(name="verify_8_5", op="attend", batch=8, n_q=32, n_kv=8, d=64, page=64, ctx=8000, new=5, ragged=True,
             window=0, sinks=0),
        # a chunk of a long prompt against what came before it
        dict(name="chunk_70b_2k_of_8k", op="attend", batch=1, n_q=64, n_kv=8, d=128, page=128, ctx=6144, new=2048,
             ragged=False, window=0, sinks=0),
        # endless chats: window of 4096 and four sinks in contexts up to 64k
        dict(name="window_decode_16", op="attend", batch=16, n_q=64, n_kv=8, d=128, page=128, ctx=65536, new=1,
             ragged=True, window=4096, sinks=4),
        # chunks of prompts under a window, wide heads
        dict(name="window_chunk_2", op="attend", batch=2, n_q=16, n_kv=8, d=256, page=64, ctx=3000, new=1500, ragged=True,
             window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    n_q, n_kv = rng.choice([(32, 32), (64, 8), (32, 8), (16, 8), (8, 1), (40, 40), (28, 4)])
    c = dict(op=rng.choice(["append", "attend", "attend", "window"]), batch=_log(rng, 1, 64), n_q=n_q, n_kv=n_kv,
             d=rng.choice([64, 96, 128, 128, 256]), page=rng.choice([64, 128, 256]), ragged=True)
    if c["op"] == "append":
        if rng.random() < 0.5:
            c.update(ctx=_log(rng, 1, 20000), new=1)
        else:
            c.update(ctx=0, new=_log(rng, 2, max(2, min(8000, 4 * 10**7 // (c["batch"] * (n_q + 2 * n_kv) * c["d"])))))
        return c
    window = 0
    if c["op"] == "window":
        window = _log(rng, 16, 8192)
        c["op"] = "attend"
    most = int((10**11 / (c["batch"] * n_q * c["d"])) ** 0.5)      # operations: no more than the largest chunk
    c["new"] = rng.choice([1, 1, rng.randint(2, 8), min(most, _log(rng, 9, 1500))])
    per = c["batch"] * n_kv * c["d"]
    ctx = _log(rng, 1, max(2, min(131072, 10**9 // per)))
    if c["new"] > 1:
        ctx = max(1, min(ctx, 5 * 10**10 // (c["batch"] * n_q * c["d"] * c["new"])))
    c.update(ctx=ctx, window=window, sinks=rng.choice([0, 1, 4, 100]) if window else 0)
    return c


def _lens(case):
    """Tokens before the call and new tokens, for each sequence: from the case alone."""
    rng = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    B, ctx, new, page = case["batch"], case["ctx"], case["new"], case["page"]
    if not case["ragged"]:
        return [ctx] * B, [new] * B
    c = [rng.randint(ctx // 8, ctx) for _ in range(B)]
    n = [rng.randint(max(1, new // 3), new) for _ in range(B)]
    if B > 1:
        c[0], n[0] = ctx, new
    if case["op"] == "append" and new == 1:
        c[-1] = ctx // page * page + page - 1      # this one fills its page
    return c, n


def _seen(case, ctx, n):
    """Cache tokens that at least one of the n queries sees, and (query, token) pairs."""
    w, s = case.get("window", 0), case.get("sinks", 0)
    if not w:
        return ctx + n, n * ctx + n * (n + 1) // 2
    first = max(0, ctx - w + 1)
    pairs = 0
    for i in range(ctx, ctx + n):
        lo = max(0, i - w + 1)
        pairs += i + 1 - lo + min(s, lo)
    return ctx + n - first + min(s, first), pairs


def work(case):
    ctx, n = _lens(case)
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    T = sum(n)
    if case["op"] == "append":
        b = T * (n_q * 4 + n_kv * 4) * d + T * 8 * d // 2          # q in and out, k and v in, angles
        for c, m in zip(ctx, n):
            total = c + m
            done = total // t - c // t                             # pages filled: codes out, their values read back
            ring = total - max(c, max(0, -(-total // t) - 2) * t)
            old = c % t if done else 0
            b += n_kv * d * (done * t * (2 + 2 + 4) + ring * 4 + old * 4)
        return {"bytes": b, "flops": 6 * T * (n_q + n_kv) * d}
    b, f = 2 * T * n_q * d * 2, 0
    for c, m in zip(ctx, n):
        seen, pairs = _seen(case, c, m)
        part = (c + m) % t                                          # the unfinished page: fp16
        part = min(part, seen)
        b += n_kv * d * ((seen - part) * 2 + part * 4)
        f += 4 * n_q * d * pairs
    return {"bytes": b, "flops": f}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    ctx, n = _lens(case)
    B, n_q, n_kv, d, t = case["batch"], case["n_q"], case["n_kv"], case["d"], case["page"]
    T = sum(n)
    rng = random.Random(seed)
    cols = max(-(-(c + m) // t) for c, m in zip(ctx, n)) + 1
    need = [-(-(c + m) // t) for c, m in zip(ctx, n)]
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    table, at = [], 0
    for k in need:
        table.append(ids[at:at + k] + [-1] * (cols - k))
        at += k
    pages, slots = len(ids), B + 1
    order = list(range(slots))
    rng.shuffle(order)
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def codes(*shape):
        x = torch.empty(shape, dtype=torch.int8, device=dev)
        for i in range(0, shape[0], 256):
            p = x[i:i + 256]
            p.copy_((torch.randn(p.shape, generator=g, device=dev) * 31).round_().clamp_(-127, 127))
        return x

    def scales():
        return 0.02 + 0.02 * torch.rand((pages, n_kv), generator=g, device=dev)

    def half(*shape):
        return torch.randn(shape, generator=g, device=dev).half()

    st = dict(case=dict(case), ctx=ctx, n=n, cu_q=i32(cu), ctx_lens=i32(ctx), table=i32(table), slots=i32(order[:B]))
    full = case["op"] == "attend"
    kshape, vshape = (n_kv, t // 64, 4, d // 16, 16, 16), (n_kv, t // 16, d, 16)
    if full:
        st["k"], st["v"] = codes(pages, *kshape), codes(pages, *vshape)
        st["ks"], st["vs"] = scales(), scales()
        st["q"] = half(T, n_q, d)
    else:
        st["k"] = torch.zeros((pages, *kshape), dtype=torch.int8, device=dev)
        st["v"] = torch.zeros((pages, *vshape), dtype=torch.int8, device=dev)
        st["ks"], st["vs"] = (torch.zeros((pages, n_kv), device=dev) for _ in range(2))
        # the projection's output: q, k and v of a token side by side
        x = half(T, (n_q + 2 * n_kv) * d)
        st["q"] = x[:, :n_q * d].view(T, n_q, d)
        st["kn"] = x[:, n_q * d:(n_q + n_kv) * d].view(T, n_kv, d)
        st["vn"] = x[:, (n_q + n_kv) * d:].view(T, n_kv, d)
        rows = max(c + m for c, m in zip(ctx, n))
        a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
            -torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
        st["rope"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
        st["pos"] = i32([c + i for c, m in zip(ctx, n) for i in range(m)])
        # the pages that this call fills, as (sequence, page of it, place in the pool)
        done = [(b, p, table[b][p]) for b in range(B) for p in range(ctx[b] // t, (ctx[b] + n[b]) // t)]
        st["done"] = i32([list(x) for x in done]).view(-1, 3)
        st["ids"] = st["done"][:, 2].contiguous()
    st["kt"], st["vt"] = half(slots, 2, *kshape), half(slots, 2, *vshape)
    if own:
        from w4a16_dequant_gemv_amd import kv
        c = kv.PagedKVCache(1, n_kv, d, 1, dev, page=t)
        c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail = (st[x] for x in ("k", "v", "ks", "vs", "kt", "vt"))
        st["cache"] = c
        st["batch"] = kv.PagedBatch(st["cu_q"], st["ctx_lens"], st["table"], st["slots"])
    return st


def _natural_k(x):
    """[..., page/64, 4, d/16, 16, 16] as [..., page, d]."""
    i, c = x.shape[-5], x.shape[-3]
    x = x.reshape(*x.shape[:-5], i, 4, c, 4, 4, 16)                 # [i][a][c][m/4][m%4][e]
    k = x.dim() - 6
    return x.permute(*range(k), k, k + 3, k + 1, k + 4, k + 2, k + 5).reshape(*x.shape[:k], i * 64, c * 16)


def _natural_v(x):
    """[..., page/16, d, 16] as [..., page, d]."""
    return x.transpose(-1, -2).reshape(*x.shape[:-3], x.shape[-3] * 16, x.shape[-2])


def _laid_k(x):
    t, d = x.shape[-2:]
    y = x.reshape(*x.shape[:-2], t // 64, 4, 4, 4, d // 16, 16)     # [i][m/4][a][m%4][c][e]
    k = y.dim() - 6
    return y.permute(*range(k), k, k + 2, k + 4, k + 1, k + 3, k + 5).reshape(*x.shape[:-2], t // 64, 4, d // 16, 16, 16)


def _laid_v(x):
    t, d = x.shape[-2:]
    return x.reshape(*x.shape[:-2], t // 16, 16, d).transpose(-1, -2)


def _to_half(x):
    """64 bits to fp16 with one rounding (a conversion by way of 32 bits would round twice)."""
    e = torch.frexp(x)[1].clamp(min=-13)
    step = torch.ldexp(torch.ones_like(x), e - 11)
    return (torch.round(x / step) * step).half()


def _rotated(x, table, pos):
    d = x.shape[-1]
    cs = table[pos.long()].double()[:, None]
    a, b = x[..., :d // 2].double(), x[..., d // 2:].double()
    return _to_half(torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1))


def _page_codes(x):
    """x [N, H, t, d] fp16 -> codes and fp32 scales [N, H]."""
    x = x.double()
    s = (x.abs().amax((-1, -2)) / 127).float().clamp(min=1e-8)
    c = torch.round((x / s.double()[..., None, None]).float()).clamp(-128, 127)
    return c, s


def _plain_append(st):
    case, cu, ctx = st["case"], st["cu_q"].long(), st["ctx_lens"].long()
    t = case["page"]
    q, k, v = _rotated(st["q"], st["rope"], st["pos"]), _rotated(st["kn"], st["rope"], st["pos"]), st["vn"]
    tok = torch.arange(k.shape[0], device=k.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    at = ctx[b] + tok - cu[b]                                       # each token's place in its sequence
    slot = st["slots"].long()
    kt, vt = _natural_k(st["kt"]), _natural_v(st["vt"])             # [slots, 2, H, t, d]
    kv_values = []
    db, dp, ids = (st["done"][:, i].long() for i in range(3))
    if db.numel():
        place = dp[:, None] * t + torch.arange(t, device=k.device)
        old = place < ctx[db][:, None]
        row = (cu[db][:, None] + place - ctx[db][:, None]).clamp(min=0)
        for new, tail, pool, scale, lay in ((k, kt, st["k"], st["ks"], _laid_k), (v, vt, st["v"], st["vs"], _laid_v)):
            x = torch.where(old[:, None, :, None], tail[slot[db], dp % 2], new[row].transpose(1, 2))
            c, s = _page_codes(x)
            pool[ids] = lay(c).to(torch.int8)
            scale[ids] = s
            kv_values.append((c * s[..., None, None]).half())
    else:
        kv_values = [k.new_empty((0, case["n_kv"], t, case["d"])) for _ in range(2)]
    total = ctx + cu[1:] - cu[:-1]
    keep = at // t >= ((total + t - 1) // t - 2)[b]                 # the last two pages stay in fp16
    bk, ak = b[keep], at[keep]
    for new, tail in ((k, kt), (v, vt)):
        tail[slot[bk], (ak // t) % 2, :, ak % t] = new[keep]
    st["kt"].copy_(_laid_k(kt))
    st["vt"].copy_(_laid_v(vt))
    return dict(q=q, k_pages=kv_values[0], v_pages=kv_values[1], k_scale=st["ks"], v_scale=st["vs"], k_tail=st["kt"],
                v_tail=st["vt"])


def _sequence(st, b, total, lo, dtype):
    """K and V of tokens [lo, total) of sequence b, [H, tokens, d]: lo is the start of a page."""
    t = st["case"]["page"]
    full = total // t
    ids = st["table"][b, lo // t:full].long()
    out = []
    for pool, scale, tail, nat in ((st["k"], st["ks"], st["kt"], _natural_k), (st["v"], st["vs"], st["vt"], _natural_v)):
        x = nat(pool[ids]).to(dtype) * scale[ids].to(dtype)[..., None, None]
        x = x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[-1])
        if total % t:
            y = nat(tail[st["slots"][b].long(), full % 2])[:, :total % t].to(dtype)
            x = torch.cat([x, y], 1)
        out.append(x)
    return out


def _plain_attend(st):
    case = st["case"]
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    G, w, s = n_q // n_kv, case["window"], case["sinks"]
    out = torch.empty_like(st["q"])
    at = 0
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["n"])):
        total = ctx + n
        lo = 0 if not w or s else max(0, ctx - w + 1) // t * t
        k, v = _sequence(st, b, total, lo, torch.float32)
        kT = k.transpose(1, 2).contiguous()
        j = torch.arange(lo, total, device=k.device)
        step = max(1, 3 * 10**8 // (n_q * (total - lo)))
        for r in range(0, n, step):
            m = min(step, n - r)
            q = st["q"][at + r:at + r + m].float().view(m, n_kv, G, d).transpose(0, 1).reshape(n_kv, m * G, d)
            x = torch.bmm(q, kT) * d ** -0.5
            i = torch.arange(ctx + r, ctx + r + m, device=k.device).repeat_interleave(G, output_size=m * G)[:, None]
            see = j <= i
            if w:
                see &= (i - j < w) | (j < s)
            x.masked_fill_(~see, float("-inf"))
            x = (x - x.amax(-1, keepdim=True)).exp_()
            o = torch.bmm(x, v) / x.sum(-1, keepdim=True)
            out[at + r:at + r + m] = o.view(n_kv, m, G, d).transpose(0, 1).reshape(m, n_q, d).half()
        at += n
    return out


def run(st):
    if st["case"]["op"] == "append":
        if own:
            c = st["cache"]
            q = c.append(st["kn"], st["vn"], st["batch"], q=st["q"], rope=st["rope"], positions=st["pos"])
            k, v = c.read(st["ids"])
            return dict(q=q, k_pages=k, v_pages=v, k_scale=c.k_scale, v_scale=c.v_scale, k_tail=c.k_tail,
                        v_tail=c.v_tail)
        return _plain_append(st)
    if own:
        return st["cache"].attend(st["q"], st["batch"], window=st["case"]["window"], sinks=st["case"]["sinks"])
    return _plain_attend(st)


def _exact_append(st):
    """Token by token and page by page, from the definition."""
    case = st["case"]
    n_kv, d, t = case["n_kv"], case["d"], case["page"]
    ang = st["rope"].double()[st["pos"].long()]
    z = torch.complex(ang[..., 0], ang[..., 1])[:, None]

    def turn(x):
        x = x.double()
        y = torch.complex(x[..., :d // 2], x[..., d // 2:]) * z
        return torch.cat([y.real, y.imag], -1)

    def stored(x):                                  # fp16 as stored, one rounding
        return torch.from_numpy(x.cpu().numpy().astype(np.float16).astype(np.float64)).to(x.device)

    new = (stored(turn(st["kn"])), st["vn"].double())
    tails = [_natural_k(st["kt"]).double(), _natural_v(st["vt"]).double()]
    scales = [st["ks"].double(), st["vs"].double()]
    values = [[], []]
    at = 0
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["n"])):
        slot = int(st["slots"][b])
        for i in range(2):
            x = new[i][at:at + n].transpose(0, 1)                   # [H, n, d]
            first = ctx // t
            if ctx % t:
                x = torch.cat([tails[i][slot, first % 2][:, :ctx % t], x], 1)
            total = ctx + n
            for p in range(first, total // t):
                y = x[:, (p - first) * t:(p - first + 1) * t]
                s = (y.abs().amax((1, 2)) / 127).float().double().clamp(min=float(torch.tensor(1e-8)))
                c = (y / s[:, None, None]).float().double().round().clamp(-128, 127)
                scales[i][int(st["table"][b, p])] = s
                values[i].append(c * s[:, None, None])
            for p in range(max(first, -(-total // t) - 2), -(-total // t)):
                lo, hi = max(p * t, ctx), min((p + 1) * t, total)
                tails[i][slot, p % 2][:, lo - p * t:hi - p * t] = x[:, lo - first * t:hi - first * t]
        at += n
    k, v = (torch.stack(x) if x else torch.empty((0, n_kv, t, d), dtype=torch.float64) for x in values)
    return dict(q=turn(st["q"]), k_pages=k, v_pages=v, k_scale=scales[0], v_scale=scales[1], k_tail=_laid_k(tails[0]),
                v_tail=_laid_v(tails[1]))


def _exact_attend(st):
    case = st["case"]
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    G, w, s = n_q // n_kv, case["window"], case["sinks"]
    rows = []
    at = 0
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["n"])):
        total = ctx + n
        j = torch.arange(total, device="cuda")
        i = ctx + torch.arange(n, device="cuda")[:, None]
        see = j <= i
        if w:
            see = see & ((j > i - w) | (j < s))
        used = see.any(0)
        ids, slot = st["table"][b, :total // t].long(), int(st["slots"][b])
        heads = []
        for h in range(n_kv):
            kv = []
            for pool, scale, tail, nat in ((st["k"], st["ks"], st["kt"], _natural_k), (st["v"], st["vs"], st["vt"], _natural_v)):
                x = nat(pool[ids, h]).double() * scale[ids, h].double()[:, None, None]
                x = torch.cat([x.reshape(-1, d), nat(tail[slot, (total // t) % 2, h])[:total % t].double()])
                kv.append(x[used])
            for m in range(G):
                q = st["q"][at:at + n, h * G + m].double()
                x = (q @ kv[0].T.contiguous()) / d ** 0.5
                p = torch.softmax(torch.where(see[:, used], x, torch.full_like(x, -torch.inf)), -1)
                heads.append(p @ kv[1])
        rows.append(torch.stack(heads, 1))
        at += n
    return torch.cat(rows)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st)
