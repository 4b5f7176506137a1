"""The paged INT8 cache as a program uses it: beside the quantized linear layers
in a captured decode step, on other streams, with drafted tokens, at sizes that
reach every way the attention is run; and what the wrappers refuse."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import w4a16_dequant_gemv_amd as w4
from gpu_util import to_dev
from test_gpu_paged import World, bits
from w4a16_dequant_gemv_amd import W4A16Error, kv

pytestmark = pytest.mark.gpu


class Layer:
    """An attention layer of quantized projections around a paged cache."""

    def __init__(self, B, n_q, n_kv, d, seed, page=64):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        hidden = n_q * d
        self.n_q, self.n_kv, self.d, self.B = n_q, n_kv, d, B
        self.qkv = w4.quantize_pack(torch.randn(((n_q + 2 * n_kv) * d, hidden), generator=g, device="cuda") * 0.06)
        self.o = w4.quantize_pack(torch.randn((hidden, hidden), generator=g, device="cuda") * 0.06)
        self.cache = kv.PagedKVCache(B * 8, n_kv, d, B, torch.device("cuda"), page=page)
        self.rope = kv.rope_table(1024, d)
        self.table = torch.arange(B * 8, dtype=torch.int32, device="cuda").view(B, 8).contiguous()
        self.slots = torch.arange(B, dtype=torch.int32, device="cuda")

    def run(self, x, batch, positions, window=0, sinks=0):
        T, hd = x.shape[0], self.n_q * self.d
        y = w4.linear(x, self.qkv)
        q, k, v = (t.view(T, -1, self.d) for t in y.split((hd, self.n_kv * self.d, self.n_kv * self.d), 1))
        q = self.cache.append(k, v, batch, q=q, rope=self.rope, positions=positions)
        a = self.cache.attend(q, batch, window=window, sinks=sinks)
        return w4.linear(a.view(T, hd), self.o), y, q, a


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_layer_against_the_definition():
    """Prompts, then single tokens: each part on the values that went into it."""
    n_q, n_kv, d, page = 8, 2, 64, 64
    layer = Layer(3, n_q, n_kv, d, 1)
    seqs = [ref.Sequence(n_kv, d, page) for _ in range(3)]
    table = layer.rope.cpu().numpy()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for n in ([100, 7, 63], [1, 1, 1], [1, 1, 1], [2, 0, 1], [1, 60, 1]):
        held = [len(s) for s in seqs]
        pos = np.concatenate([h + np.arange(m) for h, m in zip(held, n)]).astype(np.int32)
        batch = kv.PagedBatch(i32(np.concatenate([[0], np.cumsum(n)]).tolist()), i32(held), layer.table, layer.slots)
        x = (torch.randn((sum(n), n_q * d), generator=g, device="cuda") * 0.5).half()
        _, y, q, a = layer.run(x, batch, to_dev(pos))
        torch.cuda.synchronize()
        y = y.cpu().numpy().reshape(sum(n), n_q + 2 * n_kv, d)
        want_q, k = (ref.rotate(t, table, pos) for t in (y[:, :n_q], y[:, n_q:n_q + n_kv]))
        assert np.array_equal(bits(q), want_q.view(np.int16))
        at = 0
        for s, m in zip(seqs, n):
            s.append(k[at:at + m], y[at:at + m, n_q + n_kv:])
            if m:
                o, size, most = ref.attend(s, want_q[at:at + m], d ** -0.5)
                err = np.abs(a[at:at + m].cpu().numpy().astype(np.float64) - o)
                ok = bool((err <= ref.tolerance(o, size, most, len(s), d)).all())
                assert ok, (n, at)
            at += m


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_captured_decode_steps_equal_eager_ones(window, sinks):
    """One step captured, replayed with its lengths moving on, other work and
    synchronizations between the replays: every step equals the eager one."""
    B, steps = 4, 70                                           # past a page's end
    a, b = Layer(B, 8, 2, 64, 9), Layer(B, 8, 2, 64, 9)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    xs = (torch.randn((steps, B, 512), generator=g, device="cuda") * 0.5).half()
    start = [0, 5, 63, 100]
    first = (torch.randn((sum(start), 512), generator=g, device="cuda") * 0.5).half()
    cu = np.concatenate([[0], np.cumsum(start)]).tolist()
    pos0 = i32([p for n in start for p in range(n)])
    for layer in (a, b):
        layer.run(first, kv.PagedBatch(i32(cu), i32([0] * B), layer.table, layer.slots), pos0)
    want = []
    lens = i32(start)
    cu1 = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    eager = kv.PagedBatch(cu1, lens, a.table, a.slots)
    for t in range(steps):
        want.append(a.run(xs[t], eager, lens, window, sinks)[0].clone())
        lens += 1
    lens_b, x_in = i32(start), xs[0].clone()
    batch = kv.PagedBatch(cu1, lens_b, b.table, b.slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale, b.cache.k_tail, b.cache.v_tail)]
    with torch.cuda.stream(side):
        b.run(x_in, batch, lens_b, window, sinks)               # warm-up; undone below
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale, b.cache.k_tail, b.cache.v_tail), keep):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.run(x_in, batch, lens_b, window, sinks)[0]
        lens_b += 1
    for t in range(steps):
        x_in.copy_(xs[t])
        graph.replay()
        if t % 7 == 0:
            torch.cuda.synchronize()
            torch.randn(1000, device="cuda").sum().item()
        assert torch.equal(y.view(torch.int16), want[t].view(torch.int16)), t
    assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v_scale, b.cache.v_scale)


def test_two_graphs_of_one_cache():
    """Two captured calls (other batches of one cache) replayed in turn and on two
    streams: the same bits as alone."""
    w = World(4, 2, 128, 128, seed=3)
    w.append([700, 300, 129, 1000])
    x = [to_dev(w.values(2, 16)) for _ in range(2)]
    batches = [kv.PagedBatch(i32([0, 1, 2]), i32([len(s) - 1 for s in w.seqs[i:i + 2]]), to_dev(w.table[i:i + 2].copy()),
                             to_dev(w.slots[i:i + 2].copy())) for i in (0, 2)]
    want = [w.cache.attend(q, b) for q, b in zip(x, batches)]
    graphs, outs = [], []
    for q, b in zip(x, batches):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.cache.attend(q, b))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, y in zip(outs, want):
            assert torch.equal(o.view(torch.int16), y.view(torch.int16))


def test_calls_on_two_streams_at_once():
    """Appends and attention of different sequences of one cache, on two streams."""
    d, page, n_kv, n = 64, 64, 2, 150
    rng = np.random.default_rng(8)
    data = [[to_dev(rng.standard_normal((n, n_kv, d)).astype(np.float16)) for _ in range(2)] for _ in range(2)]
    q = [to_dev(rng.standard_normal((n, 8, d)).astype(np.float16)) for _ in range(2)]

    def run(streams):
        c = kv.PagedKVCache(8, n_kv, d, 2, torch.device("cuda"), page=page)
        torch.cuda.synchronize()
        outs = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                b = kv.PagedBatch(i32([0, n]), i32([0]), i32([[4 * i + j for j in range(4)]]), i32([i]))
                c.append(*data[i], b)
                outs.append(c.attend(q[i], b))
        torch.cuda.synchronize()
        return outs, c
    one = torch.cuda.current_stream()
    (a, ca), (b, cb) = run([one, one]), run([torch.cuda.Stream(), torch.cuda.Stream()])
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(ca.k, cb.k) and torch.equal(ca.v, cb.v)


def test_drafted_tokens():
    """Five drafted tokens at a time, some of them taken back: the cache goes on as
    if only the kept ones had been there."""
    w = World(3, 2, 64, 64, seed=17)
    table = ref.rope_table(600, 64)
    w.append([50, 120, 63], 8, table)
    for step in range(14):
        w.append([5, 5, 5], 8, table)
        w.attend([5, 5, 5], 8)
        for i, s in enumerate(w.seqs):
            back = (step + i) % 5
            s.k, s.v = s.k[:len(s) - back], s.v[:len(s) - back]
    w.check_storage(ring=False)
    w.attend([1, 1, 1], 8)


@pytest.mark.parametrize("d,page,n_kv,n_q,held,n", [
    (64, 64, 8, 64, [1500], [1000]),                  # eight waves a workgroup, uncut
    (128, 128, 8, 64, [1300], [1000]),
    (96, 64, 8, 64, [1200, 1040], [508, 500]),
    (128, 128, 4, 8, [4100], [2100]),                 # the same with tiles cut
    (64, 64, 8, 64, [1500], [1100]),                  # four waves, uncut
    (128, 128, 8, 64, [1300], [1030]),
    (96, 64, 8, 64, [1200, 40], [1030, 20]),
    (128, 64, 4, 8, [9000], [1100]),                  # eight waves, more than 64 tiles in a cut
    (256, 128, 2, 4, [900, 500], [600, 33]),
    (64, 128, 1, 8, [4500, 4700], [40, 30]),          # few row blocks: tiles cut and joined
    (256, 64, 1, 2, [4400], [20]),
    (128, 64, 2, 2, [5000], [70]),
    (128, 128, 1, 8, [300, 900], [5, 6]),             # 40 and 48 rows a wave
    (64, 64, 2, 16, [300, 900, 65], [5, 6, 4]),
    (96, 256, 1, 8, [700, 513], [5, 5]),
    (64, 64, 600, 600, [70], [1]),                    # more kv heads than workgroups
    (64, 64, 2, 16, [300, 200, 65], [5, 6, 4]),       # few tokens: a row block a worker, no joining
    (128, 64, 2, 4, [300, 64, 130], [1, 40, 3]),
    (96, 128, 1, 8, [300, 200], [3, 5]),
    (256, 64, 2, 4, [100, 150], [2, 3]),
    (64, 64, 1, 1024, [130, 64], [1, 2]),             # a token's heads fill several row blocks
    (128, 64, 3, 21, [200, 77], [3, 20]),             # seven heads a kv head
])
def test_every_way_the_attention_is_run(d, page, n_kv, n_q, held, n):
    w = World(len(held), n_kv, d, page, seed=sum(held), most=max(held))
    w.append(held)
    w.attend(n, n_q, front=3, back=5)
    w.attend(n, n_q, window=200, sinks=5)


@pytest.mark.parametrize("d,page,n_q,n", [(64, 128, 1, 20), (128, 128, 2, 20), (64, 128, 2, 20), (128, 128, 8, 20),
                                          (96, 256, 8, 20), (256, 128, 2, 20), (128, 128, 8, 1), (256, 256, 1, 1)])
def test_infinities_and_nan_in_masked_places(d, page, n_q, n):
    """In tokens outside the window and in tokens behind a row: the rows that do not
    see them are right, those that do are NaN.  A value that must not count is 0 in
    the definition's sequence."""
    w = World(1, 1, d, page, seed=d + n)
    L = page + 60 + n                                   # the last 60 + n tokens are in the ring
    k, v = w.values(L, 1), w.values(L, 1)
    bad = {L - n - 30: "v", L - n - 31: "k"}            # 30 tokens or more before the first row
    if n > 1:
        bad.update({L - 10: "v", L - 5: "k"})           # behind the first rows
    clean = [k.copy(), v.copy()]
    for j, which in bad.items():
        x = v if which == "v" else k
        x[j, 0, 5], x[j, 0, d - 1] = np.nan, -np.inf
        clean["kv".index(which)][j] = 0
    w.cache.append(to_dev(k), to_dev(v), w.batch([L]))
    w.seqs[0].append(*clean)
    x = w.values(n, n_q)
    out = w.cache.attend(to_dev(x), w.batch([n], ctx=[L - n]), window=30)
    torch.cuda.synchronize()
    rows = n if n == 1 else n - 10                      # rows before the first bad token behind them
    y = out.cpu().numpy().astype(np.float64)
    o, size, most = ref.attend(w.seqs[0], x, d ** -0.5, 30)
    ok = bool((np.abs(y - o)[:rows] <= ref.tolerance(o, size, most, L, d)[:rows]).all())
    assert ok
    # Row i stands at L - n + i.  A bad k makes every later row NaN; a bad v those
    # whose weight for it fp16 can hold: certainly the ones above 2^-20.
    for i in range(rows, n):
        at = L - n + i
        ks = w.seqs[0].values(0)[0][at - 29:at + 1]
        for h in range(n_q):
            e = np.exp2((ks @ x[i, h].astype(np.float64)) * d ** -0.5 / np.log(2))
            weight = e[L - 10 - (at - 29)] / e.sum()
            if at >= L - 5 or weight >= 2.0**-20:
                assert np.isnan(y[i, h]).all(), (i, h, weight)


def test_many_sequences_of_many_rows():
    """More than 64 sequences in the kernels that look them up."""
    rng = np.random.default_rng(2)
    held = rng.integers(0, 150, 140).tolist()
    n = [min(h, int(k)) for h, k in zip(held, rng.integers(0, 60, 140))]
    w = World(140, 1, 64, 64, seed=7, most=256)
    w.append(held)
    w.check_storage()
    w.attend(n, 4, front=1, back=2)
    w.attend(n, 4, window=50, sinks=2)


@pytest.mark.parametrize("d,n_kv,n_q,most", [
    (64, 2, 8, 4096),                                 # a long table: equal runs
    (64, 2, 8, 256),                                  # a short one: a row block a workgroup
    (64, 16, 64, 256),                                # and with many row blocks a wave
    (96, 8, 96, 256),
    (128, 8, 80, 256),
    (256, 8, 8, 256),
])
def test_many_sequences_of_few_rows(d, n_kv, n_q, most):
    """The same for the kernels of single and drafted tokens."""
    rng = np.random.default_rng(3)
    held = rng.integers(0, 150, 140).tolist()
    n = [min(h, int(k)) for h, k in zip(held, rng.integers(0, 4, 140))]
    w = World(140, n_kv, d, 64, seed=8, most=most)
    w.append(held)
    w.attend(n, n_q, front=1, back=2)
    w.attend(n, n_q, front=45, window=50, sinks=2)


def test_two_gib_of_queries_apart():
    """Rows 2^31 bytes and more apart: strides pass 32 bits."""
    stride = (1 << 30) + 64
    w = World(1, 1, 64, 64, seed=5)
    w.append([65])
    x = w.values(3, 4)
    big = torch.empty(2 * stride + 256, dtype=torch.float16, device="cuda")
    q = big.as_strided((3, 4, 64), (stride, 64, 1))
    q.copy_(to_dev(x))
    b = w.batch([3], ctx=[62])
    got, want = w.cache.attend(q, b), w.cache.attend(to_dev(x), b)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    k = big.as_strided((3, 1, 64), (stride, 64, 1))
    for cache_q in (q, to_dev(x)):
        w.cache.append(k if cache_q is q else k.contiguous(), k if cache_q is q else k.contiguous(),
                       w.batch([3], ctx=[65]), q=cache_q, rope=kv.rope_table(100, 64), positions=i32([65, 66, 67]))
        got = w.cache.k_tail.clone() if cache_q is q else got
    assert torch.equal(got.view(torch.int16), w.cache.k_tail.view(torch.int16))


def test_empty_calls():
    c = kv.PagedKVCache(2, 1, 64, 1, torch.device("cuda"), page=64)
    b = kv.PagedBatch(i32([0, 0]), i32([0]), i32([[0]]), i32([0]))
    x = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    assert c.append(x, x, b) is None
    assert c.append(x, x, b, q=x, rope=kv.rope_table(4, 64), positions=i32([])).shape == (0, 1, 64)
    assert c.attend(x, b).shape == (0, 1, 64)
    k, v = c.read(i32([]))
    assert k.shape == v.shape == (0, 1, 64, 64)


def test_a_replaced_tensor_is_used():
    """The cache's tensors may be replaced: the next call takes the new ones."""
    w = World(1, 1, 64, 64, seed=4)
    w.append([200])
    x, a = w.attend([1], 4)
    c = w.cache
    c.k, c.v, c.k_scale = c.k.clone(), c.v.clone(), c.k_scale.clone()
    c.v_scale, c.k_tail, c.v_tail = (t.clone() for t in (c.v_scale, c.k_tail, c.v_tail))
    c.k_tail *= 0
    b = c.attend(to_dev(x), w.batch([1], ctx=[199]))
    assert not torch.equal(a, b)
    c.k_tail = torch.zeros_like(c.k_tail).float()
    with pytest.raises(W4A16Error, match="k_tail"):
        c.attend(to_dev(x), w.batch([1], ctx=[199]))


def test_a_resized_block_table_is_used():
    """A table that the caller makes narrower or wider in place, where it is."""
    w = World(2, 2, 64, 64, seed=31)
    w.append([150, 90])
    q = to_dev(w.values(2, 4))
    pages = w.batch([1, 1]).block_table[:, :3]
    table = torch.full((2, 16), -1, dtype=torch.int32, device="cuda")
    batch = kv.PagedBatch(i32([0, 1, 2]), i32([149, 89]), table, i32(w.slots.tolist()))
    want = w.cache.attend(q, w.batch([1, 1], ctx=[149, 89]))
    for cols in (4, 16, 3):
        table.resize_(2, cols).fill_(-1)
        table[:, :3] = pages
        assert np.array_equal(bits(w.cache.attend(q, batch)), bits(want)), cols
    table.resize_(3, 4)
    with pytest.raises(W4A16Error):
        w.cache.attend(q, batch)


def test_wrappers_refuse():
    c = kv.PagedKVCache(2, 2, 64, 1, torch.device("cuda"), page=64)
    b = kv.PagedBatch(i32([0, 3]), i32([0]), i32([[0]]), i32([0]))
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    rope, pos = kv.rope_table(8, 64), i32([0, 1, 2])
    for bad in (dict(k=x.float()), dict(k=x[:, :1]), dict(k=x[:2]), dict(v=x.transpose(0, 1)), dict(k=x.cpu()),
                dict(q=x), dict(positions=pos), dict(rope=rope), dict(rope=rope, positions=pos.long()),
                dict(rope=rope, positions=pos[:2]), dict(rope=rope.double(), positions=pos),
                dict(rope=rope[:, :8].contiguous(), positions=pos), dict(rope=kv.rope_table(8, 128), positions=pos),
                dict(rope=rope[0], positions=pos), dict(rope=rope, positions=pos, q=x[:2]),
                dict(rope=rope, positions=pos, q=x[:, :1]), dict(rope=rope, positions=pos, q=x, q_out=x.float()),
                dict(k=torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda")[:, :, ::2])):
        a = dict(k=x, v=x)
        a.update(bad)
        with pytest.raises(W4A16Error):
            c.append(a.pop("k"), a.pop("v"), b, **a)
    odd = torch.zeros((3, 2 * 64 + 4), dtype=torch.float16, device="cuda")[:, :128].view(3, 2, 64)
    with pytest.raises(W4A16Error):                            # rows 8 bytes off
        c.append(odd, x, b)
    for bad in (dict(q=x.float()), dict(q=x[:, :1]), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1),
                dict(sinks=1), dict(window=4, sinks=-1), dict(window=1 << 31), dict(out=x.float()), dict(out=x[:2]),
                dict(workspace=x[:1]), dict(workspace=x.cpu()), dict(q=odd)):
        a = dict(q=x)
        a.update(bad)
        with pytest.raises(W4A16Error):
            c.attend(a.pop("q"), b, **a)
    for bad in (pos.long(), pos[None], pos.cpu(), None):
        with pytest.raises(W4A16Error):
            c.read(bad)
    for args in ((i32([0, 3, 3]), i32([0]), i32([[0]]), i32([0])), (i32([0, 3]), i32([0]).long(), i32([[0]]), i32([0])),
                 (i32([0, 3]), i32([0]), i32([0]), i32([0])), (i32([0, 3]), i32([0]), i32([[0], [1]]), i32([0])),
                 (i32([0, 3]), i32([0]), i32([[0]]), i32([0, 1])), (i32([0]), i32([]), i32([[0]]), i32([]))):
        with pytest.raises(W4A16Error):
            kv.PagedBatch(*args)
