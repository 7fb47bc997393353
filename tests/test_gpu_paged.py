"""The paged key-value cache on the GPU: block tables, append and attention
against plain 64-bit references.

Tolerances.  Tables and appended values are exact.  An attention output is a
mean of values with weights p: the scores' rounding (d products of fp32, and the
exponent's argument up to about 2^6) and the sums move it by about 2^-15 of
sum p |v|; 2^-14 is allowed, and half a unit of 2^-8 of itself where it is
rounded to bfloat16.  The log sum moves by the scores' rounding, 2^-18 of
(1 + the largest score) + 2^-14 absolute."""
import numpy as np
import pytest
import torch

import serve_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- tables

def tables(sq, ctx, new, P, free, table, capacity):
    n = len(ctx)
    t = torch.from_numpy(np.array(table, np.int32).reshape(n, -1)).cuda()
    seq, cn, cp, res = (torch.full((m,), -77, dtype=torch.int32, device="cuda") for m in (n, n + 1, n + 1, 1))
    slots = torch.full((capacity,), -77, dtype=torch.int64, device="cuda")
    sq.sq_block_tables(ints(ctx), ints(new), P, ints(free), t, seq, cn, cp, slots, res)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, seq, cn, cp, slots)] + [int(res.item())]


def check_tables(sq, ctx, new, P, free, table, capacity):
    got = tables(sq, ctx, new, P, free, table, capacity)
    want = ref.block_tables(ctx, new, P, free, table, capacity)
    for g, w, name in zip(got, want, ("table", "seq", "cu_new", "cu_pages", "slots", "result")):
        assert np.array_equal(g, w), (name, g, w)


def table_case(seed, n, top, P, new_top, spare=3, cap=0):
    rng = np.random.default_rng(seed)
    ctx = [int(x) for x in rng.integers(0, top + 1, n)]
    new = [int(x) for x in rng.integers(0, new_top + 1, n)]
    held = [-(-c // P) for c in ctx]
    total = [-(-(c + m) // P) for c, m in zip(ctx, new)]
    ids = rng.permutation(sum(total) + spare).tolist()
    stride = max(total + [1]) + 1
    table = np.full((n, stride), -5)
    pos = 0
    for i, h in enumerate(held):
        table[i, :h] = ids[pos:pos + h]
        pos += h
    return ctx, new, P, ids[pos:], table, sum(new) + cap


@pytest.mark.parametrize("n,top,P,new_top,cap", [
    (1, 0, 16, 1, 0), (1, 33, 16, 100, 5), (70, 500, 16, 1, 0), (70, 500, 32, 1, 58), (13, 200, 64, 700, 3),
    (300, 40, 128, 3, 0), (2048, 90, 16, 5, 1), (2049, 90, 16, 5, 1), (5000, 30, 256, 2, 0), (4, 9000, 256, 3000, 0)])
def test_tables(sq, n, top, P, new_top, cap):
    check_tables(sq, *table_case(n + P, n, top, P, new_top, cap=cap))


def test_tables_every_boundary(sq):
    ctx = [0, 0, 1, 15, 15, 16, 16, 17, 31, 32, 0]
    new = [0, 1, 0, 1, 2, 0, 1, 15, 1, 16, 33]
    table = np.arange(11 * 5).reshape(11, 5) + 100
    check_tables(sq, ctx, new, 16, list(range(20, 40)), table, 71)


def test_tables_report_what_is_wrong(sq):
    table = np.arange(12).reshape(3, 4)
    check_tables(sq, [16, 20, 0], [40, 3, 9], 16, [90, 91], table, 60)           # pages run out
    check_tables(sq, [16, 20, 0], [80, 3, 9], 16, list(range(50, 70)), table, 99)  # a row is full
    check_tables(sq, [16, 20, 0], [40, 3, 9], 16, list(range(50, 70)), table, 20)  # the slot map is short
    check_tables(sq, [16, -1, 0], [40, 3, -9], 16, list(range(50, 70)), table, 60)  # negative lengths
    check_tables(sq, [16, 2 ** 31 - 5, 0], [40, 9, 2], 16, list(range(50, 70)), table, 60)  # over int32
    check_tables(sq, [70, 0, 0], [3, 1, 0], 16, [], table, 9)                      # everything at once
    check_tables(sq, [3, 4, 5], [0, 0, 0], 16, [], table, 0)


def test_tables_of_no_requests(sq):
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    cn, cp, res = ints([7]), ints([7]), ints([7])
    slots = torch.full((5,), 9, dtype=torch.int64, device="cuda")
    sq.sq_block_tables(e, e, 16, e, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), e, cn, cp, slots, res)
    torch.cuda.synchronize()
    assert cn.item() == cp.item() == res.item() == 0 and slots.tolist() == [-1] * 5


def test_slots_past_32_bits(sq):
    """Page ids times the page size pass 2^31."""
    big = 2 ** 31 - 2
    check_tables(sq, [256], [300], 256, [big, big - 7], [[big - 3, 0, 0]], 300)


# ---------------------------------------------------------------- append

def plain_append(kc, vc, k, v, slots, P):
    for t, s in enumerate(slots):
        if 0 <= s < kc.shape[0] * P:
            kc[s // P, :, s % P] = k[t]
            vc[s // P, :, :, s % P] = v[t]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,d,H,n", [(16, 128, 2, 1), (16, 64, 3, 50), (32, 96, 1, 77), (64, 256, 2, 200),
                                     (128, 32, 4, 300), (256, 192, 1, 513), (16, 128, 8, 2100)])
def test_append(sq, dtype, P, d, H, n):
    g = torch.Generator().manual_seed(P + d + n)
    pages = n // P + 5
    kc = torch.randn(pages, H, P, d, generator=g).to(DT[dtype])
    vc = torch.randn(pages, H, d, P, generator=g).to(DT[dtype])
    # runs of tokens from odd places, pages in any order, some skipped or outside
    order = torch.randperm(pages, generator=g)
    flat = torch.cat([order[i] * P + torch.arange(P) for i in range(pages)])
    slots = flat[3:3 + n].clone()
    if n > 40:
        slots[20:23] = -1
        slots[30] = pages * P
        slots[31] = 2 ** 40
        cut = slots[40:].clone()
        slots[40:] = cut[torch.randperm(len(cut), generator=g)] if n < 100 else cut
    wide = torch.randn(n, 2 * H * d + 16, generator=g).to(DT[dtype])
    kd, vd, wd = kc.cuda(), vc.cuda(), wide.cuda()
    kt, vt = (wd[:, i * H * d:(i + 1) * H * d].view(n, H, d) for i in range(2))
    sq.sq_kv_append(sq.SqKvCache(kd, vd), kt, vt, slots.cuda())
    torch.cuda.synchronize()
    plain_append(kc, vc, wide[:, :H * d].reshape(n, H, d), wide[:, H * d:2 * H * d].reshape(n, H, d), slots.tolist(), P)
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,d,H,n", [(256, 256, 6, 853), (256, 256, 6, 854), (32, 96, 5, 1031), (16, 32, 12, 430)])
def test_append_around_the_larger_tiles(sq, dtype, P, d, H, n):
    test_append(sq, dtype, P, d, H, n)


# ---------------------------------------------------------------- attention

def cache(seed, lens, P, H, d, dtype, fill=0.0):
    """A fragmented cache whose places past each request's last token hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-x // P) for x in lens]
    pages = sum(need) + 2
    ids = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    k, v = torch.full((pages, H, P, d), fill), torch.full((pages, H, d, P), fill)
    pos = 0
    for r, x in enumerate(lens):
        table[r, :need[r]] = ids[pos:pos + need[r]]
        pos += need[r]
        for p in range(need[r]):
            m = min(P, x - p * P)
            k[table[r, p], :, :m] = torch.randn(H, m, d, generator=g)
            v[table[r, p], :, :, :m] = torch.randn(H, d, m, generator=g)
    return k.to(DT[dtype]), v.to(DT[dtype]), table


def attend(sq, k, v, table, lens, q, scale=None, window=0, most=None, lse=True):
    c = sq.SqKvCache(k.cuda(), v.cuda())
    n, H, d = q.shape
    most = max(list(lens) + [0]) if most is None else most
    o = torch.full((n, H, d), float("nan"), dtype=k.dtype, device="cuda")
    l = torch.full((n, H), float("nan"), device="cuda") if lse else None
    nb = sq.sq_paged_attention_workspace(c, n, H, most)
    ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device="cuda")
    sq.sq_paged_attention(c, q.cuda(), torch.from_numpy(table).cuda(), ints(list(lens)), most, o, ws, scale=scale,
                          window=window, lse=l)
    torch.cuda.synchronize()
    return o.float().cpu().numpy(), None if l is None else l.cpu().numpy()


def check_attend(sq, k, v, table, lens, q, scale=None, window=0, most=None):
    o, l = attend(sq, k, v, table, lens, q, scale, window, most)
    sc = q.shape[2] ** -0.5 if scale is None else scale
    kk, vv = (torch.nan_to_num(x.float(), 0.0, 0.0, 0.0).numpy() for x in (k, v))
    wo, wl, mag = ref.attention(q.float().numpy(), kk, vv, table, list(lens), sc, window)
    assert np.isfinite(o).all()
    lim = 2.0 ** -14 * mag + (2.0 ** -8 * np.abs(wo) if k.dtype == torch.bfloat16 else 0.0)
    assert (np.abs(o - wo) <= lim).all(), float((np.abs(o - wo) / np.maximum(lim, 1e-30)).max())
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l), empty) and not o[empty].any()
    e = np.abs(l[~empty] - wl[~empty])
    assert (e <= 2.0 ** -14 + 2.0 ** -18 * (1 + np.abs(wl[~empty]))).all(), e.max()
    return o


def queries(seed, n, H, d, dtype):
    return torch.randn(n, H, d, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 64])
def test_attention_lengths(sq, dtype, d, P):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]
    k, v, t = cache(d + P, lens, P, 2, d, dtype, fill=float("nan"))
    check_attend(sq, k, v, t, lens, queries(d, len(lens), 6, d, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 1), (33, 3), (64, 2)])
def test_attention_head_groups(sq, dtype, H, Hkv):
    lens = [300, 7, 0]
    k, v, t = cache(H, lens, 32, Hkv, 64, dtype, fill=float("inf"))
    check_attend(sq, k, v, t, lens, queries(H, 3, H, 64, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 129, 1000, 5000])
def test_attention_windows(sq, dtype, window):
    lens = [0, 1, 33, 128, 513, 1200]
    k, v, t = cache(window, lens, 16, 1, 64, dtype)
    check_attend(sq, k, v, t, lens, queries(window, len(lens), 4, 64, dtype), window=window)


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("bf16", 256), ("f32", 128)])
def test_attention_long(sq, dtype, P):
    """Many splits, requests of very different lengths, a loose max_len."""
    lens = [20011, 3, 0, 9000]
    k, v, t = cache(P, lens, P, 1, 128, dtype)
    q = queries(3, 4, 3, 128, dtype)
    a = check_attend(sq, k, v, t, lens, q)
    b = check_attend(sq, k, v, t, lens, q, most=60000)
    assert np.allclose(a, b, rtol=2.0 ** -7, atol=1e-3)


def test_attention_of_many_requests(sq):
    """More (request, head) units than workgroups wanted: one split each."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 300, 700)]
    k, v, t = cache(9, lens, 16, 3, 32, "bf16", fill=float("nan"))
    check_attend(sq, k, v, t, lens, queries(5, 700, 6, 32, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_pages_that_are_not_there(sq, dtype):
    """Table entries outside the cache are absent tokens, also all of them."""
    lens = [100, 64, 40, 3000]
    k, v, t = cache(6, lens, 16, 2, 64, dtype)
    t[0, 2], t[0, 6] = -1, 10 ** 6
    t[1, :] = -1
    t[3, 10:150] = 2 ** 31 - 1
    check_attend(sq, k, v, t, lens, queries(6, 4, 4, 64, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_scores_far_apart(sq, dtype):
    """One key wins by far, early or late; scale 0 and a negative scale."""
    lens = [700, 700]
    k, v, t = cache(8, lens, 16, 1, 64, dtype)
    q = queries(8, 2, 2, 64, dtype)
    k[t[0, 0], 0, 3] = 30 * q[0, 0]
    k[t[1, 43], 0, 5] = 30 * q[1, 1]
    for scale in (None, 0.0, -0.3, 1.0):
        o, l = attend(sq, k, v, t, lens, q, scale)
        sc = 0.125 if scale is None else scale
        wo, wl, mag = ref.attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), t, lens, sc, 0)
        # scores reach thousands here: their rounding, 2^-22 of the largest, moves the weights
        slack = 2.0 ** -22 * (1 + np.abs(wl).max()) * 8
        lim = (2.0 ** -14 + slack) * mag + 2.0 ** -8 * np.abs(wo)
        assert (np.abs(o - wo) <= lim).all()
        assert (np.abs(l - wl) <= 2.0 ** -14 + 2.0 ** -18 * (1 + np.abs(wl))).all()


def test_attention_takes_length_limits(sq):
    """seq_lens above max_len or above the table's row are cut; below zero is empty."""
    k, v, t = cache(10, [90, 90, 90], 16, 1, 64, "bf16")
    q = queries(10, 3, 2, 64, "bf16")
    o, l = attend(sq, k, v, t, [90, 10 ** 6, -4], q, most=90)
    wo, wl, mag = ref.attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), t, [90, 90, 0], 0.125, 0)
    assert (np.abs(o - wo) <= 2.0 ** -14 * mag + 2.0 ** -8 * np.abs(wo)).all() and np.isneginf(l[2]).all()
    o, _ = attend(sq, k, v, t[:, :2].copy(), [90, 20, 0], q, most=90)
    wo, _, mag = ref.attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), t, [32, 20, 0], 0.125, 0)
    assert (np.abs(o - wo) <= 2.0 ** -14 * mag + 2.0 ** -8 * np.abs(wo)).all()


@pytest.mark.parametrize("dtype,P,window", [("bf16", 16, 0), ("bf16", 64, 70), ("f32", 128, 0)])
def test_attention_with_any_max_len(sq, dtype, P, window):
    """The largest max_len: the table's rows bound the lengths, and the workspace."""
    lens = [1000, 1, 0, 700]
    k, v, t = cache(20 + P, lens, P, 2, 64, dtype)
    q = queries(20, 4, 4, 64, dtype)
    c = sq.SqKvCache(k.cuda(), v.cuda())
    o, lse = torch.empty(4, 4, 64, dtype=k.dtype, device="cuda"), torch.empty(4, 4, device="cuda")
    room = sq.sq_paged_attention_workspace(c, 4, 4, t.shape[1] * P)
    ws = torch.empty(max(room, 16), dtype=torch.uint8, device="cuda")
    sq.sq_paged_attention(c, q.cuda(), torch.from_numpy(t).cuda(), ints(lens), 2 ** 31 - 1, o, ws[:room],
                          window=window, lse=lse)
    wo, wl, mag = ref.attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), t, lens, 0.125, window)
    lim = 2.0 ** -14 * mag + (2.0 ** -8 * np.abs(wo) if dtype == "bf16" else 0.0)
    assert (np.abs(o.float().cpu().numpy() - wo) <= lim).all()
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.isneginf(wl))


def test_attention_strided_queries_streams_and_graph(sq):
    lens = [400, 30, 1]
    k, v, t = cache(12, lens, 16, 2, 128, "bf16")
    q = queries(12, 3, 4, 128, "bf16")
    want, _ = attend(sq, k, v, t, lens, q)
    wide = torch.zeros(3, 4 * 128 + 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 128:640] = q.view(3, 512).cuda()
    qs = wide[:, 128:640].view(3, 4, 128)
    c = sq.SqKvCache(k.cuda(), v.cuda())
    table, ln = torch.from_numpy(t).cuda(), ints(lens)
    o = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sq.sq_paged_attention_workspace(c, 3, 4, 400), dtype=torch.uint8, device="cuda")
    call = lambda: sq.sq_paged_attention(c, qs, table, ln, 400, o, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert np.array_equal(o.float().cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        ln.copy_(ints([400 - 13 * i, 30 + i, i]))
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, o)


def test_a_window_needs_no_more_workspace(sq):
    """A workspace made for (n, max_len) serves smaller calls and any window."""
    c = sq.SqKvCache(torch.zeros(4, 3, 16, 64, device="cuda"), torch.zeros(4, 3, 64, 16, device="cuda"))
    for n, most in ((1, 20000), (7, 5000), (90, 3001), (700, 130)):
        room = sq.sq_paged_attention_workspace(c, n, 6, most)
        ws = torch.empty(max(room, 16), dtype=torch.uint8, device="cuda")
        for m in {1, n // 2 + 1, n}:
            q = torch.zeros(m, 6, 64, device="cuda")
            table, lens, o = torch.zeros(m, 1, dtype=torch.int32, device="cuda"), ints([5] * m), torch.empty_like(q)
            for ln in {1, 100, 129, 1000, 1100, most // 3, most - 1, most}:
                if ln <= most:
                    for w in (0, 1, 500, ln):
                        sq.sq_paged_attention(c, q, table, lens, ln, o, ws[:room], window=w)
    torch.cuda.synchronize()


def test_cache_past_32_bit_offsets(sq):
    """A cache of more than 2^31 elements: pages at its far end."""
    pages, H, P, d = 70000, 2, 128, 128
    k = torch.empty(pages, H, P, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(pages, H, d, P, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 31
    c = sq.SqKvCache(k, v)
    n = 200
    g = torch.Generator().manual_seed(2)
    kt, vt, q = (torch.randn(n, H, d, generator=g).bfloat16(), torch.randn(n, H, d, generator=g).bfloat16(),
                 torch.randn(1, 4, d, generator=g).bfloat16())
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, x // P]) * P + x % P for x in range(n)])
    sq.sq_kv_append(c, kt.cuda(), vt.cuda(), slots.cuda())
    o = torch.empty(1, 4, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, sq.sq_paged_attention_workspace(c, 1, 4, n)), dtype=torch.uint8, device="cuda")
    sq.sq_paged_attention(c, q.cuda(), table.cuda(), ints([n]), n, o, ws)
    torch.cuda.synchronize()
    small_k = k[pages - 2:].float().cpu().numpy()[::-1]
    small_v = v[pages - 2:].float().cpu().numpy()[::-1]
    assert np.array_equal(small_k[0][:, :, :], kt[:P].float().numpy().transpose(1, 0, 2))
    wo, _, mag = ref.attention(q.float().numpy(), small_k, small_v, [[0, 1]], [n], d ** -0.5, 0)
    assert (np.abs(o.float().cpu().numpy() - wo) <= 2.0 ** -14 * mag + 2.0 ** -8 * np.abs(wo)).all()
