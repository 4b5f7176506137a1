"""The paged INT8 cache from its definition, in 64 bits with numpy: what the
pages, the ring and attention over them have to be.  Sequences are plain lists
of tokens here; only `page_order` knows the order inside a page."""
import numpy as np


def to_half(x):
    """binary64 to fp16, one rounding."""
    with np.errstate(over="ignore"):
        return np.asarray(x, np.float64).astype(np.float16)


def rope_table(rows, dim, base=10000.0):
    a = np.arange(rows, dtype=np.float64)[:, None] * base ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x, table, positions, interleaved=False):
    """fp16 x [T, heads, d] rotated to `positions`, as fp16."""
    y = x.astype(np.float64)
    half = table.shape[1]
    bad = (positions < 0) | (positions >= table.shape[0])
    cs = table.astype(np.float64)[np.where(bad, 0, positions)][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    a[bad] = b[bad] = np.nan
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a, b
    else:
        y[..., :half], y[..., half:2 * half] = a, b
    return to_half(y)


def quantize(x):
    """fp16 page x [t, d] -> int8 codes, fp32 scale."""
    x = x.astype(np.float32)
    s = np.float32(max(np.float32(np.abs(x).max() / np.float32(127)), np.float32(1e-8)))
    return np.clip(np.rint(x / s), -128, 127).astype(np.int8), s


def page_order(x, which):
    """[t, d] in the order of tokens -> the flat order of a page."""
    t, d = x.shape
    out = np.empty(t * d, x.dtype)
    tok, ch = np.meshgrid(np.arange(t), np.arange(d), indexing="ij")
    if which == "k":
        i, r = tok // 64, tok % 64
        m, a = r // 16 * 4 + r % 4, r % 16 // 4
        at = ((((i * 4 + a) * (d // 16) + ch // 16) * 16) + m) * 16 + ch % 16
    else:
        at = (tok // 16 * d + ch) * 16 + tok % 16
    out[at] = x
    return out


class Sequence:
    """The tokens of one sequence: k (rotated) and v, fp16 [tokens, n_kv, d]."""

    def __init__(self, n_kv, d, page):
        self.page = page
        self.k = np.zeros((0, n_kv, d), np.float16)
        self.v = np.zeros((0, n_kv, d), np.float16)

    def append(self, k, v):
        self.k, self.v = np.concatenate([self.k, k]), np.concatenate([self.v, v])

    def __len__(self):
        return len(self.k)

    def values(self, h, hidden=()):
        """K and V of head h as attention sees them, binary64, and which tokens
        are there at all (pages in `hidden` are not)."""
        t, total = self.page, len(self)
        k, v = self.k[:, h].astype(np.float64), self.v[:, h].astype(np.float64)
        there = np.ones(total, bool)
        for p in range(total // t):
            for x in (k, v):
                c, s = quantize(x[p * t:(p + 1) * t].astype(np.float16))
                x[p * t:(p + 1) * t] = c.astype(np.float64) * np.float64(s)
            if p in hidden:
                there[p * t:(p + 1) * t] = False
        return k, v, there


def attend(seq, q, scale, window=0, sinks=0, hidden=(), quant=None):
    """q fp16 [n, n_q, d], the last n tokens' queries -> (o, sum p|v|, the largest
    scale * sum|q k|), binary64 [n, n_q, d], [n, n_q, d] and a number."""
    n, n_q, d = q.shape
    n_kv = seq.k.shape[1]
    total = len(seq)
    i = total - n + np.arange(n)[:, None]
    j = np.arange(total)[None]
    see = j <= i
    if window:
        see &= (i - j < window) | (j < sinks)
    out, size, most = np.zeros((n, n_q, d)), np.zeros((n, n_q, d)), 0.0
    for h in range(n_kv):
        k, v, there = seq.values(h, hidden)
        ok = see & there
        k, v = np.where(there[:, None], k, 0), np.where(there[:, None], v, 0)
        for g in range(n_q // n_kv):
            x = q[:, h * (n_q // n_kv) + g].astype(np.float64)
            s = np.where(ok, scale * (x @ k.T), -np.inf)
            most = max(most, float((scale * np.abs(x) @ np.abs(k).T).max(initial=0)))
            m = np.where(ok.any(1, keepdims=True), s.max(1, keepdims=True), 0)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p = np.where(l > 0, p / np.where(l > 0, l, 1), 0)
            out[:, h * (n_q // n_kv) + g] = p @ v
            size[:, h * (n_q // n_kv) + g] = p @ np.abs(v)
    return out, size, most


def tolerance(o, size, most, tokens, d, weights=2.0**-11):
    """How far the kernel may be off, by its roundings: o to fp16 (2^-11), each
    weight to fp16 (2^-11 of sum p|v|; WEIGHTS_IN_TWO where it is two parts), scores in
    binary32 (d products and a few
    steps, each 2^-24 of the largest score's terms, counted for numerator and
    denominator), sums over the tokens and the hardware exponential (2^-20)."""
    rel = weights + 2 * (d + 8) * 2.0**-24 * most + 2 * (tokens + 64) * 2.0**-24 + 2.0**-20
    return 2.0**-11 * np.abs(o) + rel * size + 2.0**-25


# A weight as two fp16 parts: what the second leaves is half a step of its own, 2^-11 of
# at most 2^-11 of the weight, or 2^-25 where it is below fp16's normal numbers, of a
# largest weight of 2^10 or more: 2^-35 for each of up to 2^13 tokens.
WEIGHTS_IN_TWO = 2.0**-22 + 2.0**-22


def balanced(n_kv, d, tokens):
    """K, V [tokens, n_kv, d], a query [1, n_kv, d] and a scale, for which half of the
    tokens nearly cancel the other half, so that an output shows how exact the weights
    are: its own rounding is small beside them.  K holds whole numbers with a scale of 1
    and the query does not see its largest channel, so scores are exact."""
    k = np.zeros((tokens, n_kv, d))
    k[::16, :, 0] = 127
    k[1::2, :, 1] = 16
    q = np.zeros((1, n_kv, d))
    q[0, :, 1] = 1 + np.arange(n_kv)
    scale = 1 / 64
    ratio = np.exp(-q[0, :, 1] * 16 * scale)[:, None]            # weight of an even token over an odd one's
    v = np.where(np.arange(tokens)[:, None, None] % 2 == 0, np.ones((n_kv, d)), -ratio)
    return k.astype(np.float16), v.astype(np.float16), q.astype(np.float16), scale
