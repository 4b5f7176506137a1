"""Microscaled 4-bit floating point (MXFP4: quantisation and the product of two
quantised operands) and attention over the paged 8-bit KV cache for sequences that
share a long prefix, as cases that can be timed.

MXFP4: 32 consecutive values of a row share a scale 2^(s - 127), s a byte (255 is NaN);
a value is a code of 4 bits, sign, two exponent bits and one of mantissa, which stands
for 0, 0.5, 1, 1.5, 2, 3, 4 or 6 times the scale.  s = floor(log2(largest |x|)) - 2 + 127.
Codes lie two in a byte, the even one in its low half; block b's scale of a row is at
[b // 8][row][b % 8], zeros behind the last.

Paged cache: a page holds `page` tokens of one sequence, for every kv head, as int8 codes
with one fp32 scale per (page, head) for K and one for V.  The last two pages of a
sequence are also kept in fp16 (the ring); a page that is not full yet is read from
there.  Inside a page, K lies as [page/64][4][d/16][16][16] (token 64*i + 16*(m/4) + 4*a +
m%4 of channel 16*c + e at [i][a][c][m][e]) and V as [page/16][d][16].  The sequences
of a group have their first pages in common: the same pool pages in their block tables.
"""
import json
import random

import torch

own = False

# Layer shapes: 7B has 4096 channels, 11008 between, 32 heads of 128 channels each with
# its own K and V; 70B 8192 and 28672, 64 query heads on 8 kv heads.


def listed():
    return [
        # activations of a serving step, 64 tokens of the 70B layout: latency
        dict(name="quant_act_64", op="quant", rows=64, k=8192, stride=8192, type="float16"),
        # activations of a chunk of prompts: the gate's half of a fused projection's output, an odd number of tokens
        dict(name="quant_act_odd", op="quant", rows=2047, k=11008, stride=22016, type="bfloat16"),
        # the largest weight of a 70B layer
        dict(name="quant_weight_70b", op="quant", rows=28672, k=8192, stride=8192, type="float32"),
        # one token through a 7B projection: latency
        dict(name="linear_7b_1", op="linear", m=1, n=4096, k=4096, type="float16"),
        # a serving step of 8 sequences through the widest layer of the 70B layout
        dict(name="linear_70b_8", op="linear", m=8, n=28672, k=8192, type="float16"),
        # a serving step of 333 sequences: more rows than a decode kernel holds, fewer than fill the card; odd sizes
        dict(name="linear_odd_333", op="linear", m=333, n=5003, k=5024, type="bfloat16"),
        # a prompt of 2048 tokens through a 7B layer
        dict(name="linear_7b_2048", op="linear", m=2048, n=11008, k=4096, type="float16"),
        # packed prompts through the widest layer of the 70B layout
        dict(name="linear_70b_7999", op="linear", m=7999, n=28672, k=8192, type="float16"),
        # four answers to one short instruction on the 7B layout: latency
        dict(name="prefix_7b_4", op="prefix", batch=4, groups=1, n_q=32, n_kv=32, d=128, page=128, prefix=512, own=100,
             new=1),
        # a serving step: 64 chats behind one system prompt, each with its own history
        dict(name="prefix_70b_64", op="prefix", batch=64, groups=1, n_q=64, n_kv=8, d=128, page=128, prefix=4096,
             own=1000, new=1),
        # five drafted tokens of 40 sequences behind three different instructions; small heads and pages
        dict(name="prefix_groups_40_5", op="prefix", batch=40, groups=3, n_q=32, n_kv=8, d=64, page=64, prefix=2000,
             own=700, new=5),
        # 32 questions about one long document
        dict(name="prefix_70b_32_128k", op="prefix", batch=32, groups=1, n_q=64, n_kv=8, d=128, page=128, prefix=131072,
             own=500, new=1),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "prefix", "prefix"])
    if op == "quant":
        k = 32 * _log(rng, 1, 512)
        rows = _log(rng, 1, min(30000, 2 * 10**8 // k))
        return dict(op=op, rows=rows, k=k, stride=k * rng.choice([1, 1, 2]), type=rng.choice(["float16", "bfloat16", "float32"]))
    if op == "linear":
        n, k = _log(rng, 64, 30000), 32 * _log(rng, 2, 512)
        m = rng.choice([1, rng.randint(2, 16), rng.randint(17, 256), _log(rng, 257, 8000)])
        return dict(op=op, m=min(m, max(1, 18 * 10**11 // (n * k))), n=n, k=k, type=rng.choice(["float16", "float16", "bfloat16"]))
    n_q, n_kv = rng.choice([(32, 32), (64, 8), (32, 8), (16, 8), (8, 1), (40, 40), (28, 4)])
    batch, page, d = _log(rng, 1, 128), rng.choice([64, 128, 256]), rng.choice([64, 96, 128, 128, 256])
    new = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 60)])
    most = min(131072, 3 * 10**8 // (n_kv * d), 34 * 10**9 // (batch * new * n_q * d))
    own_most = min(4000, 3 * 10**8 // (batch * n_kv * d), 4 * 10**8 // (batch * new * n_q))
    return dict(op=op, batch=batch, groups=min(batch, rng.choice([1, 1, 2, 5])), n_q=n_q, n_kv=n_kv, d=d, page=page,
                prefix=_log(rng, page, max(most, 2 * page)), own=_log(rng, 1, max(2, own_most)), new=new)


def _lens(case):
    """From the case alone: sequences of each group, its shared pages, and each sequence's
    tokens before the call and new ones."""
    rng = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    B, G, page = case["batch"], case["groups"], case["page"]
    cuts = [0] + sorted(rng.sample(range(1, B), G - 1)) + [B]
    most = max(1, case["prefix"] // page)
    pages = [most] + [rng.randint(max(1, most // 8), most) for _ in range(G - 1)]
    ctx, new = [], []
    for g in range(G):
        for _ in range(cuts[g], cuts[g + 1]):
            ctx.append(pages[g] * page + rng.randint(case["own"] // 8, case["own"]))
            new.append(rng.randint(max(1, case["new"] // 3), case["new"]))
    return cuts, pages, ctx, new


def work(case):
    if case["op"] == "quant":
        n, size = case["rows"] * case["k"], 4 if case["type"] == "float32" else 2
        return {"bytes": n * 2 * size + n // 32, "flops": 4 * n}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k // 2 + n * k // 32 + 2 * m * n, "flops": 2 * m * n * k}
    cuts, pages, ctx, new = _lens(case)
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    b = 2 * sum(new) * n_q * d * 2 + sum(pages) * t * n_kv * d * 2
    f = 0
    for g, p in enumerate(pages):
        for c, m in zip(ctx[cuts[g]:cuts[g + 1]], new[cuts[g]:cuts[g + 1]]):
            mine, part = c + m - p * t, (c + m) % t
            b += n_kv * d * ((mine - part) * 2 + part * 4)
            f += 4 * n_q * d * (m * c + m * (m + 1) // 2)
    return {"bytes": b, "flops": f}


# The values that the codes of 4 bits stand for, without their sign.
STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _scale_of(x):
    """The exponent of each block's scale, int32 [rows, blocks], of x [rows, blocks, 32] fp32: one of 128 is NaN."""
    top = x.abs().amax(-1)
    e = (torch.frexp(top)[1] - 3).clamp(min=-127)                   # frexp's mantissa is below 1
    return torch.where(top == 0, -127, torch.where(torch.isfinite(top), e, 128))


def _rounded(x):
    """x [rows, k] as the values of its MXFP4 form, fp32, and the scales' bytes."""
    y = x.float().view(x.shape[0], -1, 32)
    e = _scale_of(y)
    at = e.clamp(max=127)[..., None]
    a = torch.ldexp(y, (-at // 2)).ldexp_(-at - (-at // 2))          # in two steps: 2^127 and more has no fp32 value
    mag = a.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_(-6, 6)
    v = torch.ldexp(a, at // 2).ldexp_(at - at // 2)
    v = torch.where(e[..., None] == 128, float("nan"), v)
    return v.view(x.shape), (e + 127).to(torch.uint8)


def _packed(w):
    """Codes and scales of w [rows, k], as a program keeps a quantised weight."""
    codes, scales = [], []
    for part in w.split(4096):
        v, s = _rounded(part)
        a = torch.ldexp(v.view(*s.shape, 32), 127 - s[..., None].int()).view(v.shape)
        mag = a.abs()
        c = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
        c |= (a < 0).to(torch.uint8) << 3
        codes.append(c[:, ::2] | c[:, 1::2] << 4)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def _values(codes, scales):
    """Codes [rows, k/2] and scales [rows, k/32] as fp32 [rows, k]."""
    table = torch.tensor(STEPS + tuple(-x for x in STEPS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).view(*scales.shape, 32)
    return torch.ldexp(table[c.int()], scales[..., None].int() - 127).view(codes.shape[0], -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    if case["op"] == "quant":
        # activations have a few large channels; weights are small and even
        rows, k = case["rows"], case["stride"]
        x = torch.randn((rows, k), generator=g, device=dev)
        x *= 0.02 if case["type"] == "float32" else torch.where(torch.rand(k, generator=g, device=dev) < 0.01, 40.0, 1.0)
        return dict(case=dict(case), x=x.to(getattr(torch, case["type"]))[:, :case["k"]])
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn((m, k), generator=g, device=dev)
        x *= torch.where(torch.rand(k, generator=g, device=dev) < 0.01, 20.0, 1.0)
        codes, scales = _packed(torch.randn((n, k), generator=g, device=dev) * 0.02)
        st = dict(case=dict(case), x=x.to(getattr(torch, case["type"])), codes=codes, scales=scales)
        if own:
            from w4a16_dequant_gemv_amd import mxfp4
            st["weight"] = mxfp4.MXTensor.from_blocks(codes, scales)
        return st

    cuts, pages, ctx, new = _lens(case)
    B, n_q, n_kv, d, t = case["batch"], case["n_q"], case["n_kv"], case["d"], case["page"]
    rng = random.Random(seed)
    need = [-(-(c + m) // t) for c, m in zip(ctx, new)]
    cols = max(need) + 1
    total = sum(pages) + sum(need) - sum(p * (b - a) for p, a, b in zip(pages, cuts, cuts[1:]))
    ids = list(range(total + 3))
    rng.shuffle(ids)
    at, table = 0, []
    for i, p in enumerate(pages):
        shared, at = ids[at:at + p], at + p
        for b in range(cuts[i], cuts[i + 1]):
            mine = need[b] - p
            table.append(shared + ids[at:at + mine] + [-1] * (cols - need[b]))
            at += mine
    slots = list(range(B + 1))
    rng.shuffle(slots)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def codes8(*shape):
        x = torch.empty(shape, dtype=torch.int8, device=dev)
        for i in range(0, shape[0], 256):
            p = x[i:i + 256]
            p.copy_((torch.randn(p.shape, generator=g, device=dev) * 31).round_().clamp_(-127, 127))
        return x

    kshape, vshape = (n_kv, t // 64, 4, d // 16, 16, 16), (n_kv, t // 16, d, 16)
    st = dict(case=dict(case), cuts=cuts, pages=pages, ctx=ctx, new=new, cu_q=i32(cu), ctx_lens=i32(ctx),
              table=i32(table), slots=i32(slots[:B]), cu_seqs=i32(cuts), shared=i32(pages))
    st["k"], st["v"] = codes8(len(ids), *kshape), codes8(len(ids), *vshape)
    st["ks"], st["vs"] = (0.02 + 0.02 * torch.rand((len(ids), n_kv), generator=g, device=dev) for _ in range(2))
    st["kt"], st["vt"] = (torch.randn((B + 1, 2, *s), generator=g, device=dev).half() for s in (kshape, vshape))
    st["q"] = torch.randn((cu[-1], n_q, d), generator=g, device=dev).half()
    if own:
        from w4a16_dequant_gemv_amd import kv
        c = kv.PagedKVCache(1, n_kv, d, 1, dev, page=t)
        c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail = (st[x] for x in ("k", "v", "ks", "vs", "kt", "vt"))
        st["cache"] = c
        st["batch"] = kv.PagedBatch(st["cu_q"], st["ctx_lens"], st["table"], st["slots"])
        st["prefix"] = kv.SharedPrefix(st["cu_seqs"], st["shared"], max(pages))
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


def _plain_prefix(st):
    """Group by group: every query on the shared pages, then on its own sequence's tokens
    (padded to the longest), one softmax over both."""
    case = st["case"]
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    G = n_q // n_kv
    dev = st["q"].device
    out = torch.empty_like(st["q"])
    pools = ((st["k"], st["ks"], st["kt"], _natural_k), (st["v"], st["vs"], st["vt"], _natural_v))
    at = 0
    for i, p in enumerate(st["pages"]):
        lo, hi = st["cuts"][i], st["cuts"][i + 1]
        ctx, new = st["ctx_lens"][lo:hi].long(), (st["cu_q"][lo + 1:hi + 1] - st["cu_q"][lo:hi]).long()
        B, N, T = hi - lo, max(st["new"][lo:hi]), sum(st["new"][lo:hi])
        pad = max(c + m for c, m in zip(st["ctx"][lo:hi], st["new"][lo:hi])) // t + 1 - p       # pages of their own
        total = ctx + new
        ids = st["table"][lo, :p].long()
        cols = torch.arange(p, p + pad, device=dev)
        mine = st["table"][lo:hi].long()[:, cols.clamp(max=st["table"].shape[1] - 1)].clamp(min=0)
        ring = (cols == (total // t)[:, None])                                               # the unfinished page
        both = []
        for pool, scale, tail, nat in pools:
            x = nat(pool[ids]).float() * scale[ids][..., None, None]                         # [p, H, t, d]
            y = nat(pool[mine]).float() * scale[mine][..., None, None]                       # [B, pad, H, t, d]
            z = nat(tail[st["slots"][lo:hi].long()])[:, cols % 2].float()
            y = torch.where(ring[..., None, None, None], z, y)
            both.append((x.transpose(0, 1).reshape(n_kv, p * t, d),
                         y.transpose(1, 2).reshape(B * n_kv, pad * t, d)))
        # rows of a group: [kv head, token, query head]; of a sequence, padded: [sequence, kv head, token, query head]
        q = st["q"][at:at + T].float().view(T, n_kv, G, d)
        seq = torch.repeat_interleave(torch.arange(B, device=dev), new, output_size=T)
        tok = torch.arange(T, device=dev) - (st["cu_q"][lo:hi].long() - at)[seq]
        s1 = torch.bmm(q.transpose(0, 1).reshape(n_kv, T * G, d), both[0][0].transpose(1, 2).contiguous())
        qp = q.new_zeros((B, N, n_kv, G, d))
        qp[seq, tok] = q
        s2 = torch.bmm(qp.transpose(1, 2).reshape(B * n_kv, N * G, d), both[0][1].transpose(1, 2).contiguous())
        s2 = s2.view(B, n_kv, N, G, pad * t)[seq, :, tok]                                    # [T, H, G, tokens]
        hidden = torch.arange(p * t, (p + pad) * t, device=dev) > (ctx[seq] + tok)[:, None]
        s2 = (s2 * d ** -0.5).masked_fill_(hidden[:, None, None], float("-inf"))
        s1 = s1.view(n_kv, T, G, -1).mul_(d ** -0.5)
        m = torch.maximum(s1.amax(-1).transpose(0, 1), s2.amax(-1))                          # [T, H, G]
        p1, p2 = s1.sub_(m.transpose(0, 1)[..., None]).exp_(), (s2 - m[..., None]).exp_()
        l = p1.sum(-1).transpose(0, 1) + p2.sum(-1)
        o = torch.bmm(p1.view(n_kv, T * G, -1), both[1][0]).view(n_kv, T, G, d).transpose(0, 1)
        pp = p2.new_zeros((B, N, n_kv, G, pad * t))
        pp[seq, tok] = p2
        v2 = torch.where(torch.arange(p * t, (p + pad) * t, device=dev)[:, None] < total[:, None, None, None],
                         both[1][1].view(B, n_kv, pad * t, d), 0.0).view(B * n_kv, pad * t, d)
        o = o + torch.bmm(pp.transpose(1, 2).reshape(B * n_kv, N * G, -1), v2).view(B, n_kv, N, G, d)[seq, :, tok]
        out[at:at + T] = (o / l[..., None]).reshape(T, n_q, d).half()
        at += T
    return out


def run(st):
    op = st["case"]["op"]
    if op == "quant":
        x = st["x"]
        if own:
            from w4a16_dequant_gemv_amd import mxfp4
            q = mxfp4.quantize(x)
            return dict(values=mxfp4.dequantize(q, dtype=x.dtype), scales=q.scales)
        v, s = _rounded(x)
        s = torch.nn.functional.pad(s, (0, -s.shape[1] % 8)).view(s.shape[0], -1, 8).transpose(0, 1).contiguous()
        return dict(values=v.to(x.dtype), scales=s)
    if op == "linear":
        if own:
            from w4a16_dequant_gemv_amd import mxfp4
            return mxfp4.linear(st["x"], st["weight"])
        x, _ = _rounded(st["x"])
        return torch.matmul(x, _values(st["codes"], st["scales"]).t()).to(st["x"].dtype)
    if own:
        return st["cache"].attend(st["q"], st["batch"], prefix=st["prefix"])
    return _plain_prefix(st)


def _exact_rounded(x):
    """x's MXFP4 values in binary64, and its scales' bytes, from the definition."""
    y = x.double().reshape(x.shape[0], -1, 32)
    top = y.abs().amax(-1)
    e = torch.floor(torch.log2(top.clamp(min=2.0**-200)))
    e += (torch.exp2(e + 1) <= top).double()
    e -= (torch.exp2(e) > top).double()
    e = (e - 2).clamp(min=-127)
    unit = torch.exp2(e)[..., None]
    y /= unit
    mag = y.abs()
    # a border between two values belongs to the one whose mantissa bit is 0
    index = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        index += (mag >= border) if up else (mag > border)
    value = torch.tensor(STEPS, dtype=torch.float64, device=y.device)[index.long()]
    return (value * torch.sign(y) * unit).reshape(x.shape), (e + 127).to(torch.uint8)


def _exact_values(codes, scales):
    low, high = codes.long() % 16, codes.long() // 16
    c = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = low, high
    v = torch.tensor(STEPS, dtype=torch.float64, device=c.device)[c % 8] * (1.0 - 2.0 * (c // 8))
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _exact_prefix(st):
    """Sequence by sequence over its whole block table, from the definition."""
    case = st["case"]
    n_q, n_kv, d, t = case["n_q"], case["n_kv"], case["d"], case["page"]
    G = n_q // n_kv
    rows = []
    at = 0
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["new"])):
        total = ctx + n
        see = torch.arange(total, device="cuda") <= ctx + torch.arange(n, device="cuda")[:, None]
        ids, slot = st["table"][b, :total // t].long(), int(st["slots"][b])
        heads = []
        for h in range(n_kv):
            kv = []
            for pool, scale, tail, nat in ((st["k"], st["ks"], st["kt"], _natural_k), (st["v"], st["vs"], st["vt"], _natural_v)):
                x = nat(pool[ids, h]).double() * scale[ids, h].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, d), nat(tail[slot, (total // t) % 2, h])[:total % t].double()]))
            q = st["q"][at:at + n, h * G:(h + 1) * G].double().transpose(0, 1).reshape(G * n, d)
            x = (q @ kv[0].T.contiguous()).view(G, n, total) / d ** 0.5
            p = torch.softmax(torch.where(see, x, torch.full_like(x, -torch.inf)), -1)
            heads.append((p.view(G * n, total) @ kv[1]).view(G, n, d).transpose(0, 1))
        rows.append(torch.cat(heads, 1))
        at += n
    return torch.cat(rows)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "quant":
        v, s = zip(*(_exact_rounded(p) for p in st["x"].split(2048)))
        return dict(values=torch.cat(v), scales=None)
    if case["op"] == "linear":
        x, _ = _exact_rounded(st["x"])
        return torch.cat([x @ _exact_values(c, s).T.contiguous() for c, s in zip(st["codes"].split(4096), st["scales"].split(4096))], 1)
    return _exact_prefix(st)
