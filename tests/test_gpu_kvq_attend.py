"""sq_kvq_attention against 64 bits: single tokens, prompts and mixtures of
them, over caches whose places outside the requests hold rubbish (bytes that are
NaN as e4m3, scales that are NaN, infinite or negative)."""
import math

import numpy as np
import pytest
import torch

import kvq_reference as ref

pytestmark = pytest.mark.gpu
FMT = ["int8", "e4m3"]
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(seed, n, H, d, dtype):
    return torch.randn(n, H, d, generator=torch.Generator().manual_seed(seed)).to(ref.DT[dtype])


def run(sq, c, q, table, lens, new=None, scale=None, window=0, most=None, pad=0):
    """o, lse as float64, rows past the last query checked to be left as they were."""
    dev = c if isinstance(c, sq.SqKvqCache) else c.gpu(sq)
    n, H, d = q.shape
    qd = torch.cat([q, q.new_zeros(pad, H, d)]).cuda()
    cu = None if new is None else ints([0] + np.cumsum(new).tolist())
    most = max(list(lens) + [0]) if most is None else most
    o = torch.full((n + pad, H, d), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n + pad, H), 77.0, device="cuda")
    nb = sq.sq_kvq_attention_workspace(dev, len(lens), n + pad, H, most)
    ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device="cuda")
    sq.sq_kvq_attention(dev, qd, torch.from_numpy(table).cuda(), ints(list(lens)), most, o, ws, cu_q=cu, scale=scale,
                        window=window, lse=lse)
    torch.cuda.synchronize()
    assert (o[n:] == 77).all() and (lse[n:] == 77).all()
    return o[:n].cpu().double(), lse[:n].cpu().double()


def check(sq, c, q, table, lens, new=None, scale=None, window=0, most=None, pad=0):
    o, lse = run(sq, c, q, table, lens, new, scale, window, most, pad)
    cu = list(range(len(lens) + 1)) if new is None else [0] + np.cumsum(new).tolist()
    sc = q.shape[2] ** -0.5 if scale is None else scale
    w = ref.attention(c, q, table, lens, cu, sc, window, 2 ** 31 if most is None else most)
    lo, ll = ref.limits(w, "bf16" if q.dtype == torch.bfloat16 else "f32")
    assert torch.isfinite(o).all()
    off = (o - w[0]).abs()
    assert (off <= lo).all(), float((off / lo.clamp(min=1e-30)).max())
    none = torch.isneginf(w[1])
    assert torch.equal(torch.isneginf(lse), none) and not o[none].any()
    off = (lse - w[1]).abs()[~none]
    assert (off <= ll[~none]).all(), float((off / ll[~none]).max())
    return o, lse


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 64])
def test_token_lengths(sq, fmt, dtype, d, P):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]
    c, t = ref.filled(lens, P, 2, d, fmt, d + P)
    check(sq, c, queries(d, len(lens), 6, d, dtype), t, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 1), (33, 3), (64, 2)])
def test_token_head_groups(sq, dtype, H, Hkv):
    lens = [300, 7, 0]
    c, t = ref.filled(lens, 32, Hkv, 64, "e4m3", H)
    check(sq, c, queries(H, 3, H, 64, dtype), t, lens)
    check(sq, c, queries(H, 3, H, 64, dtype), t, lens, new=[1, 1, 1])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 129, 1000, 5000])
def test_token_windows(sq, fmt, window):
    lens = [0, 1, 33, 128, 513, 1200]
    c, t = ref.filled(lens, 16, 1, 64, fmt, window)
    check(sq, c, queries(window, len(lens), 4, 64, "bf16"), t, lens, window=window)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("P", [16, 256])
def test_token_long(sq, fmt, P):
    """Many splits, lengths far apart, a loose max_len, a request cut to max_len."""
    lens = [20011, 3, 0, 9000]
    c, t = ref.filled(lens, P, 1, 128, fmt, P)
    q = queries(3, 4, 3, 128, "bf16")
    check(sq, c, q, t, lens)
    check(sq, c, q, t, lens, most=60000)
    check(sq, c, q, t, lens, most=5000)


def test_token_of_many_requests(sq):
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 300, 700)]
    c, t = ref.filled(lens, 16, 3, 32, "e4m3", 9)
    check(sq, c, queries(5, 700, 6, 32, "bf16"), t, lens)


# ---------------------------------------------------------------- prompts

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 128])
def test_prompts(sq, fmt, dtype, d, P):
    """Whole prompts and turns behind a context: tiles of 128 rows and 64 tokens that are full, begin and
    end anywhere; requests of one token and of none among them."""
    new = [43, 0, 1, 64, 130, 17, 2, 200]
    ctx = [0, 5, 64, 63, 1, 300, 90, 128]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, P, 2, d, fmt, d + P)
    check(sq, c, queries(d, sum(new), 6, d, dtype), t, lens, new=new, pad=9)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (8, 1), (15, 1), (16, 1), (17, 1), (130, 1), (40, 2)])
def test_prompt_head_groups(sq, H, Hkv):
    """Also groups of more heads than a tile has rows."""
    new, ctx = [19, 1, 70, 2], [3, 40, 0, 64]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, Hkv, 64, "int8", H)
    check(sq, c, queries(H, sum(new), H, 64, "bf16"), t, lens, new=new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 127, 300, 10 ** 6])
def test_prompt_windows(sq, dtype, window):
    new, ctx = [150, 3, 400, 1], [0, 200, 77, 500]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 32, 2, 64, "e4m3", window % 1000)
    check(sq, c, queries(window % 1000, sum(new), 6, 64, dtype), t, lens, new=new, window=window)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("new,ctx", [([33], [6000]), ([5, 70], [9000, 2000]), ([2, 3], [3000, 5]), ([300], [0]),
                                     ([1], [4000]), ([8], [513]), ([128, 1, 1], [1500, 3000, 0])])
def test_prompt_splits(sq, fmt, new, ctx):
    """Few tiles behind long contexts are split over them and joined; one request of any size."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 1, 128, fmt, sum(new))
    for dtype in ("bf16", "f32"):
        check(sq, c, queries(1, sum(new), 4, 128, dtype), t, lens, new=new, pad=3)
    check(sq, c, queries(2, sum(new), 4, 128, "bf16"), t, lens, new=new, window=700)


@pytest.mark.parametrize("new", [[1], [3], [40], [0]])
def test_capacity_larger_than_the_queries(sq, new):
    """As a captured graph has it: room for 500 queries, few there."""
    lens = [1000]
    c, t = ref.filled(lens, 64, 2, 64, "int8", 5)
    check(sq, c, queries(4, sum(new), 4, 64, "bf16"), t, lens, new=new, pad=500 - sum(new))


@pytest.mark.parametrize("window", [0, 90])
def test_requests_longer_than_the_bound(sq, window):
    """Positions from max_len on, or past the table, are not seen; queries keep their places."""
    new, ctx = [300, 1, 40], [100, 399, 500]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 32, 2, 64, "int8", 15)
    q = queries(4, sum(new), 4, 64, "bf16")
    for most in (0, 1, 33, 250, 399, 512):
        check(sq, c, q, t, lens, new=new, window=window, most=most)
    t = np.ascontiguousarray(t[:, :10])
    check(sq, c, q, t, lens, new=new, window=window)  # the reference knows rows that end


def test_more_queries_than_tokens(sq):
    """The first queries of such a request stand before its first token: nothing to see."""
    new, lens = [10, 90, 4], [3, 40, 0]
    c, t = ref.filled(lens, 16, 1, 64, "e4m3", 5)
    o, lse = check(sq, c, queries(4, sum(new), 3, 64, "bf16"), t, lens, new=new)
    assert torch.isneginf(lse[:7]).all() and torch.isneginf(lse[10:60]).all() and torch.isneginf(lse[100:]).all()


def test_prompt_of_many_requests(sq):
    g = np.random.default_rng(3)
    new, ctx = g.integers(0, 40, 300).tolist(), g.integers(0, 100, 300).tolist()
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 1, 32, "int8", 9)
    check(sq, c, queries(5, sum(new), 2, 32, "bf16"), t, lens, new=new)


def test_long_prompt(sq):
    new, ctx = [2100, 700], [0, 1300]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 64, 1, 128, "int8", 9)
    check(sq, c, queries(5, sum(new), 4, 128, "bf16"), t, lens, new=new)


# ---------------------------------------------------------------- both forms

BOTH = [([1, 1, 1, 1], [99, 63, 39, 2999]), ([40, 64, 40, 900], [60, 0, 0, 2100])]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx", BOTH)
def test_pages_that_are_not_there(sq, fmt, dtype, new, ctx):
    """Table entries outside the cache are absent tokens, also all of them."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 2, 64, fmt, 6)
    t[0, 2], t[0, 6] = -1, 10 ** 6
    t[1, :] = -1
    t[3, 10:150] = 2 ** 31 - 1
    check(sq, c, queries(6, sum(new), 4, 64, dtype), t, lens, new=new)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("new,ctx", BOTH)
@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_scales_far_apart(sq, fmt, new, ctx, spread):
    """Value scales over 2^(+-spread): the reference of the probabilities grows on the way, small blocks count
    for what they are.  Keys' scales are kept near each other (a softmax has one maximum)."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 1, 64, fmt, 7, spread=spread)
    c.scales[..., 0] = torch.where(c.held.view(c.pages, 1, -1, 16).any(-1), 1 / 64, c.scales[..., 0])
    for dtype in ("bf16", "f32"):
        check(sq, c, queries(6, sum(new), 4, 64, dtype), t, lens, new=new)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx", BOTH)
def test_scores_far_apart(sq, fmt, dtype, new, ctx):
    """Sharp and flat softmaxes, scale 0 and a negative scale; queries of very different sizes."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 32, 2, 64, fmt, 8)
    q = queries(8, sum(new), 4, 64, dtype)
    for scale in (0.0, -0.125, 3.0, 1e-30):
        check(sq, c, q, t, lens, new=new, scale=scale)
    for up in (1e-30, 1e-6, 20.0):
        check(sq, c, q * up, t, lens, new=new)
    q[:, 1] = 0
    q[:, 2, 5] *= 2.0 ** 20
    check(sq, c, q, t, lens, new=new, scale=2.0 ** -20)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx", BOTH)
def test_queries_that_are_not_finite(sq, fmt, dtype, new, ctx):
    """NaN in whole rows that meet it, the others' bits as they were."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 2, 64, fmt, 9)
    q = queries(9, sum(new), 6, 64, dtype)
    o, lse = run(sq, c, q, t, lens, new)
    hit = torch.zeros(sum(new), 6, dtype=torch.bool)
    q[0, 1, 9], q[-1, 4, 0], q[2, 0, 63] = NAN, INF, -INF
    hit[0, 1] = hit[-1, 4] = hit[2, 0] = True
    o2, lse2 = run(sq, c, q, t, lens, new)
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx", BOTH)
def test_scores_past_the_range(sq, dtype, new, ctx):
    """Every score +inf, or -inf: no softmax.  Some of -inf beside finite ones: they weigh nothing."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 1, 64, "int8", 10)
    held = c.held[:, None, :, None].expand_as(c.k)
    c.k[held] = 128 + 100
    c.scales[..., 0] = torch.where(c.held.view(c.pages, 1, -1, 16).any(-1), 1e6, c.scales[..., 0])
    q = queries(9, sum(new), 4, 64, dtype)
    q[:, 0], q[:, 1] = 1e36, -1e36
    o, lse = run(sq, c, q, t, lens, new)
    assert torch.isnan(o[:, :2]).all() and torch.isnan(lse[:, :2]).all()
    # keys of zero among them: scores of zero beside -inf
    for r in (0, 3):
        for x in range(0, lens[r], 7):
            c.k[t[r, x // 16], :, x % 16] = 128
    cu = [0] + np.cumsum(new).tolist()
    o, lse = run(sq, c, q, t, lens, new)
    for r in (0, 3):
        for i in range(cu[r], cu[r + 1]):
            own = lens[r] - new[r] + i - cu[r]
            x = np.arange(0, own + 1, 7)
            pg = torch.from_numpy(t[r][x // 16]).long()
            val = (ref.code_values(c.v[pg, 0, 0, :, x % 16], "int8")
                   * c.scales[pg, 0, 0, 1].double()[:, None])
            want, mag = val.mean(0), val.abs().mean(0)
            lim = (2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * want.abs()
            assert ((o[i, 1] - want).abs() <= lim).all()
            assert abs(float(lse[i, 1]) - math.log(len(x))) <= 2.0 ** -13
        assert torch.isnan(o[cu[r]:cu[r + 1], 0]).all()


@pytest.mark.parametrize("new,ctx", BOTH)
def test_queries_inside_a_wider_buffer(sq, new, ctx):
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 2, 96, "e4m3", 11)
    n, H, d = sum(new), 4, 96
    wide = torch.randn(n, 3 * H * d + 8, generator=torch.Generator().manual_seed(1)).bfloat16()
    q = wide[:, H * d:2 * H * d].unflatten(1, (H, d))
    o, lse = run(sq, c, q.contiguous(), t, lens, new)
    dev, w = c.gpu(sq), wide.cuda()
    o2 = torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sq.sq_kvq_attention_workspace(dev, len(lens), n, H, max(lens)), dtype=torch.uint8, device="cuda")
    sq.sq_kvq_attention(dev, w[:, H * d:2 * H * d].unflatten(1, (H, d)), torch.from_numpy(t).cuda(), ints(lens), max(lens),
                        o2, ws, cu_q=ints([0] + np.cumsum(new).tolist()))  # and without a log sum
    assert torch.equal(o2.cpu().double(), o)


def test_offsets_outside_the_queries(sq):
    """cu_q that falls, is negative or passes the queries: guards stay, the call ends."""
    lens = [100, 200, 30, 64]
    c, t = ref.filled(lens, 16, 1, 64, "int8", 12)
    dev = c.gpu(sq)
    q, o = queries(3, 80, 2, 64, "bf16").cuda(), torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, sq.sq_kvq_attention_workspace(dev, 4, 80, 2, 200)), dtype=torch.uint8, device="cuda")
    for cu in ([0, 20, -7, 10 ** 9, 30], [2 ** 31 - 1] * 5, [-2 ** 31, 0, 0, 20, 80], [80, 60, 20, 10, 0]):
        sq.sq_kvq_attention(dev, q, torch.from_numpy(t).cuda(), ints(lens), 200, o[:80], ws, cu_q=ints(cu))
        torch.cuda.synchronize()
        assert (o[80:] == 7).all()


def test_workspaces_of_smaller_calls(sq):
    """One workspace of the largest call serves every smaller one."""
    dev = ref.Cache(1, 2, 16, 64, "int8").gpu(sq)
    rng = np.random.default_rng(1)
    for _ in range(300):
        n, nq, most = int(rng.integers(1, 200)), int(rng.integers(1, 5000)), int(2 ** rng.uniform(0, 20))
        big = sq.sq_kvq_attention_workspace(dev, n, nq, 12, most)
        n2, q2, m2 = int(rng.integers(1, n + 1)), int(rng.integers(1, nq + 1)), int(rng.integers(0, most + 1))
        assert sq.sq_kvq_attention_workspace(dev, n2, q2, 12, m2) <= big


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype,d,window", [("bf16", 128, 0), ("bf16", 64, 200), ("bf16", 96, 0), ("f32", 64, 0),
                                            ("f32", 96, 100), ("f32", 32, 0), ("bf16", 32, 0), ("f32", 128, 0)])
def test_prompts_that_fill_the_card(sq, fmt, dtype, d, window):
    """Enough rows for the larger tiles, unsplit; a request of few queries and one of none among them, and
    pages that do not exist."""
    new, ctx = [700, 2, 0, 331], [37, 100, 5, 0]
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 8, d, fmt, d)
    t[0, 20:23] = -1
    check(sq, c, queries(d, sum(new), 64, d, dtype), t, lens, new=new, window=window, pad=5)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("new,ctx", BOTH)
def test_scales_of_zero(sq, fmt, new, ctx):
    """A cache made elsewhere may hold blocks of zeros with a scale of zero: their values are zero and their
    tokens count, their keys' scores are zero.  All values of one request are."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, 2, 64, fmt, 13)
    for r, n in enumerate(lens):
        for i, x in enumerate(range(0, n, 16)):
            if i % 3 == 1 or r == 1:
                c.scales[t[r, x // 16], :, :, 1] = 0.0
            if i % 4 == 2:
                c.scales[t[r, x // 16], :, :, 0] = 0.0
    for dtype in ("bf16", "f32"):
        check(sq, c, queries(6, sum(new), 4, 64, dtype), t, lens, new=new)


# ---------------------------------------------------------------- prompts behind long contexts, wide heads

# Tiles hold more rows there: four ragged requests of few rows, and many rows at once.
LONG = [([40, 0, 64, 56], [60, 5, 0, 2100], 4, 1), ([640, 2, 0, 421], [37, 100, 5, 700], 256, 16)]


def long_table(t, P, span=4500):
    """The table with room for more positions, whose pages do not exist."""
    return np.concatenate([t, np.full((t.shape[0], -(-span // P)), -1, t.dtype)], 1)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("new,ctx,H,Hkv", LONG)
@pytest.mark.parametrize("P", [16, 128])
def test_larger_tiles(sq, fmt, new, ctx, H, Hkv, P):
    """Ragged requests, one without new tokens, pages that do not exist, value scales far apart."""
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, P, Hkv, 128, fmt, 17, spread=8.0)
    c.scales[..., 0] = torch.where(c.held.view(c.pages, 1, -1, 16).any(-1), 1 / 64, c.scales[..., 0])
    t = long_table(t, P)
    q = queries(17, sum(new), H, 128, "bf16")
    check(sq, c, q, t, lens, new=new, most=4400, pad=2)
    t[0, 0] = -1
    t[3, 256 // P:512 // P] = 10 ** 6
    check(sq, c, q, t, lens, new=new, most=4400, scale=-0.2)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("new,ctx,window", [([40], [6000], 4500), ([33], [9000], 0), ([64], [6900], 4096),
                                            ([50, 60], [5000, 4100], 4200)])
def test_larger_tiles_behind_long_contexts(sq, fmt, new, ctx, window):
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 32, 2, 128, fmt, 19)
    check(sq, c, queries(19, sum(new), 8, 128, "bf16"), t, lens, new=new, window=window)


@pytest.mark.parametrize("new,ctx,H,Hkv", LONG)
def test_larger_tiles_of_queries_that_are_not_finite(sq, new, ctx, H, Hkv):
    lens = [a + b for a, b in zip(ctx, new)]
    c, t = ref.filled(lens, 16, Hkv, 128, "int8", 21)
    t = long_table(t, 16)
    q = queries(21, sum(new), H, 128, "bf16")
    o, lse = run(sq, c, q, t, lens, new, most=4400)
    hit = torch.zeros(sum(new), H, dtype=torch.bool)
    q[0, 1, 9], q[-1, 3, 0], q[2, 0, 127] = NAN, INF, -INF
    hit[0, 1] = hit[-1, 3] = hit[2, 0] = True
    o2, lse2 = run(sq, c, q, t, lens, new, most=4400)
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def test_prompts_of_pages_past_32_bits(sq):
    """The same bits from pages whose bytes begin past 2^32, in both forms and tile sizes."""
    lens, new, P, Hkv, d = [4500, 70], [40, 33], 256, 2, 128
    c, t = ref.filled(lens, P, Hkv, d, "int8", 23)
    dev = c.gpu(sq)
    pages = 2 ** 32 // (P * Hkv * d) + c.pages
    big = sq.SqKvqCache(*(torch.zeros(pages, *x.shape[1:], dtype=x.dtype, device="cuda")
                          for x in (dev.k, dev.v, dev.scales)))
    for a, b in ((big.k, dev.k), (big.v, dev.v), (big.scales, dev.scales)):
        a[pages - c.pages:] = b
    for dtype in ("bf16", "f32"):
        q = queries(23, sum(new), 8, d, dtype)
        for n, m in ((new, q), ([1, 1], q[:2])):
            o, lse = run(sq, dev, m, t, lens, n)
            o2, lse2 = run(sq, big, m, t + (pages - c.pages), lens, n)
            assert torch.equal(o, o2) and torch.equal(lse, lse2) and o.abs().max() > 0
