"""The 8-bit cache as a server uses it: in the hybrid loop, in captured graphs,
on other streams."""
import numpy as np
import pytest
import torch

import kvq_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def read_back(sq, m):
    """Every request's keys and values as the cache stands for them, float64 on the CPU."""
    lens = m.ctx.tolist()
    cu = [0] + np.cumsum(lens).tolist()
    k = torch.empty(cu[-1], m.cache.n_kv_heads, 128, device="cuda")
    v = torch.empty_like(k)
    sq.sq_kvq_load(m.cache, m.table, ints(cu), k, v)
    return [(k[a:b].cpu().double(), v[a:b].cpu().double()) for a, b in zip(cu, cu[1:])]


def plain(q, k, v):
    """o and sum p |v| of queries [m][H][d] at the last positions of k, v [n][kv][d]."""
    m, H, n, G = q.shape[0], q.shape[1], k.shape[0], q.shape[1] // k.shape[1]
    seen = torch.arange(n) <= (n - m + torch.arange(m))[:, None]
    x = torch.einsum("mhd,nhd->hmn", q.double(), k.repeat_interleave(G, 1)) * q.shape[2] ** -0.5
    p = torch.softmax(x.masked_fill(~seen, -torch.inf), -1)
    vv = v.repeat_interleave(G, 1)
    return torch.einsum("hmn,nhd->mhd", p, vv), torch.einsum("hmn,nhd->mhd", p, vv.abs())


def near(got, want):
    o, mag = want
    lim = (2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * o.abs()  # a weight's 11 bits, fp32 scores and sums, bfloat16
    assert ((got.cpu().double() - o).abs() <= lim).all()


@pytest.mark.parametrize("kv_cache", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_hybrid(sq, kv_cache, page):
    """Prompts, tokens, a further prompt, tokens: attention over what the cache stands for, which is near
    the keys and values that went in, and the recurrent layer's outputs as beside a plain cache."""
    from quantized_recurrent_state_gated_amd import hybrid as H
    n, heads, qh, kvh = 3, 2, 6, 2
    turns = [[70, 1, 33], [1] * 3, [1] * 3, [20, 5, 0], [1] * 3, [1] * 3, [1] * 3]
    make = lambda c: H.HybridLayers(n, heads, [32] * heads, qh, kvh, page, 160, kv_cache=c)  # noqa: E731
    m, other = make(kv_cache), make("plain")
    m.cache.k.fill_(0xff), m.cache.v.fill_(0x7f), m.cache.scales.fill_(float("nan"))  # whatever was there
    gen = torch.Generator(device="cuda")
    gen.manual_seed(page)
    came = [([], []) for _ in range(n)]
    for lens in turns:
        x = H.activations(sum(lens), heads, qh, kvh, gen)
        at = [0] + np.cumsum(lens).tolist()
        if lens == [1] * 3:
            o, a = m.token(x)
            o2, _ = other.token(x)
        else:
            o, a = m.prompts(lens, x)
            o2 = other.prompts(lens, {k: t for k, t in x.items() if k != "aq"})
        assert torch.equal(o, o2)
        held = read_back(sq, m)
        for r in range(n):
            mine = slice(at[r], at[r + 1])
            came[r][0].append(x["ak"][mine].cpu().double())
            came[r][1].append(x["av"][mine].cpu().double())
            if lens[r]:
                near(a[mine], plain(x["aq"][mine].cpu(), *held[r]))
    for r in range(n):
        for back, went in zip(held[r], came[r]):
            went = torch.cat(went)
            # each of up to 6 calls that wrote into a block moves a value by half a step (of 127 or, next to
            # the largest, of 14) of the block's largest value, and the block's largest is at most the head's
            step = went.abs().amax((0, 2), keepdim=True) / (127 if kv_cache == "int8" else 14)
            assert ((back - went).abs() <= 6 * step / 2 * (1 + 2.0 ** -10)).all()


def test_hybrid_command():
    """The module's own command, small."""
    import json
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-m", "quantized_recurrent_state_gated_amd.hybrid", "--requests", "2", "--prompt", "40",
                        "--steps", "3", "--heads", "2", "--kv-cache", "int8"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert json.loads(r.stdout.strip().splitlines()[-1])["kv_cache"] == "int8"


class Side:
    """Cache, tables and outputs of a server with room for n requests, N new tokens a call."""

    def __init__(self, sq, n, N, most, fmt, kv=2, qh=8, d=128, P=16):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.sq, self.n, self.P, self.most, cols = sq, n, P, most, -(-most // P)
        self.cache = ref.Cache(n * cols, kv, P, d, fmt, seed=1).gpu(sq)
        self.table, self.seq = torch.full((n, cols), -1, **i32), torch.zeros(n, **i32)
        self.cu, self.cp, self.res = (torch.zeros(m, **i32) for m in (n + 1, n + 1, 1))
        self.slots = torch.zeros(N, dtype=torch.int64, device="cuda")
        self.o = torch.zeros(N, qh, d, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(N, qh, device="cuda")
        self.ko, self.vo = (torch.zeros(N, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        nb = sq.sq_kvq_attention_workspace(self.cache, n, N, qh, most)
        self.ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")

    def call(self, x, ctx, new, free, stream=None, ws=None):
        sq = self.sq
        sq.sq_block_tables(ctx, new, self.P, free, self.table, self.seq, self.cu, self.cp, self.slots, self.res, stream=stream)
        sq.sq_kvq_append(self.cache, x[0], x[1], ctx, self.cu, self.table, stream=stream)
        sq.sq_kvq_attention(self.cache, x[2], self.table, self.seq, self.most, self.o, self.ws if ws is None else ws,
                            cu_q=self.cu, lse=self.lse, stream=stream)
        sq.sq_kvq_load(self.cache, self.table, self.cu, self.ko, self.vo, first=ctx, stream=stream)

    def out(self):
        used = int(self.cu[-1])
        return [t.clone() for t in (self.table, self.seq, self.cu, self.o[:used], self.lse[:used], self.ko[:used],
                                    self.vo[:used], self.cache.k)]


def new_tokens(N, seed, kv=2, qh=8, d=128):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda h: torch.randn(N, h, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    return r(kv), r(kv), r(qh)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,N", [(3, 600), (1, 90)])
def test_graph(sq, fmt, n, N):
    """Tables, append, attention and read-back in one graph, replayed for other lengths (whole prompts, single
    tokens, nothing) with eager work between, bit for bit as the same calls made eagerly."""
    most = 3000
    i32 = dict(dtype=torch.int32, device="cuda")
    a, b = Side(sq, n, N, most, fmt), Side(sq, n, N, most, fmt)
    ctx, new = torch.zeros(n, **i32), torch.zeros(n, **i32)
    per = -(-most // 16)
    free = torch.randperm(n * per, device="cuda").to(torch.int32)
    x = new_tokens(N, 3)
    for side in (a, b):  # once outside a capture
        side.call(x, ctx, new, free)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call(x, ctx, new, free)
    for step, lens in enumerate(([N // n] * n, [1] * n, [N - 2 * n] + [0] * (n - 1), [0] * n, [5] + [1] * (n - 1))):
        new.copy_(ints(lens))
        graph.replay()
        b.call(x, ctx, new, free)
        torch.cuda.synchronize()
        for x1, x2 in zip(a.out(), b.out()):
            assert torch.equal(x1, x2)
        assert int(a.res) == 0 and int(a.cu[-1]) == sum(lens)
        taken = int(a.cp[-1])
        free.copy_(torch.cat([free[taken:], free[:taken]]))
        ctx.copy_(a.seq)
        for t in x:
            t.mul_(-1.125)


def test_two_graphs_of_one_workspace(sq):
    """Replayed in turn: nothing is kept in the workspace between calls."""
    c, t = ref.filled([2500, 900], 16, 2, 128, "int8", 3)
    dev, tab = c.gpu(sq), torch.from_numpy(t).cuda()
    lens, q = ints([2500, 900]), new_tokens(70, 5)[2]
    cu = ints([0, 69, 70])
    ws = torch.empty(sq.sq_kvq_attention_workspace(dev, 2, 70, 8, 2500), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.zeros(2, 8, 128, device="cuda").bfloat16(), torch.zeros_like(q)

    def one():
        sq.sq_kvq_attention(dev, q[:2], tab, lens, 2500, o1, ws)

    def many():
        sq.sq_kvq_attention(dev, q, tab, lens, 2500, o2, ws, cu_q=cu)

    one(), many()
    torch.cuda.synchronize()
    want = o1.clone(), o2.clone()
    graphs = []
    for f in (one, many):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for order in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0)):
        o1.zero_(), o2.zero_()
        for i in order:
            graphs[i].replay()
        ws.fill_(0xff)
        torch.cuda.synchronize()
        assert torch.equal(o1, want[0]) and torch.equal(o2, want[1])


def test_streams(sq):
    """On the current stream, on one given, and two servers on two streams at once."""
    n, N = 2, 300
    i32 = dict(dtype=torch.int32, device="cuda")
    sides = [Side(sq, n, N, 1000, "int8") for _ in range(4)]
    ctx, new = torch.zeros(n, **i32), ints([200, 100])
    free = torch.randperm(n * 63, device="cuda").to(torch.int32)
    x = new_tokens(N, 9)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sides[0].call(x, ctx, new, free)
    with torch.cuda.stream(s1):
        sides[1].call(x, ctx, new, free)
    sides[2].call(x, ctx, new, free, stream=s1)
    sides[3].call(x, ctx, new, free, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for s in sides[1:]:
        for x1, x2 in zip(sides[0].out(), s.out()):
            assert torch.equal(x1, x2)


def test_attention_agrees_with_the_plain_cache(sq):
    """Keys and values whose codes hold them exactly: both caches, one answer."""
    g = torch.Generator().manual_seed(2)
    lens, P, H, d = [300, 17, 1], 32, 2, 64
    table, pages = ref.tables(lens, P, g)
    N = sum(lens)
    x = torch.randint(-127, 128, (2, N, H, d), generator=g).float()
    x[:, :, :, 0] = 127.0  # every token's largest: the scale is one
    k, v = (t.bfloat16().cuda() for t in x / 64)
    tab, cu = torch.from_numpy(table).cuda(), [0] + np.cumsum(lens).tolist()
    c8 = ref.Cache(pages, H, P, d, "int8").gpu(sq)
    sq.sq_kvq_append(c8, k, v, ints([0] * 3), ints(cu), tab)
    c16 = sq.SqKvCache(torch.zeros(pages, H, P, d, device="cuda").bfloat16(), torch.zeros(pages, H, d, P, device="cuda").bfloat16())
    slots = torch.tensor([int(table[r, i // P]) * P + i % P for r in range(3) for i in range(lens[r])], device="cuda")
    sq.sq_kv_append(c16, k, v, slots)
    q = torch.randn(3, 6, d, generator=g).bfloat16().cuda()
    o8, o16 = torch.empty_like(q), torch.empty_like(q)
    l8, l16 = torch.empty(3, 6, device="cuda"), torch.empty(3, 6, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    sq.sq_kvq_attention(c8, q, tab, ints(lens), 300, o8, ws, lse=l8)
    sq.sq_paged_attention(c16, q, tab, ints(lens), 300, o16, ws, lse=l16)
    # two roundings to bfloat16, and the weights' 11 bits of values up to 2
    assert ((o8 - o16).float().abs() <= 2.0 ** -7 * o16.float().abs() + 2.0 ** -9).all()
    assert ((l8 - l16).abs() <= 2.0 ** -13).all()
