"""sq_kvq_attention where weights, value scales and scores lie far apart."""
import numpy as np
import pytest
import torch

import kvq_reference as ref
import kvq_weights as kw
from test_gpu_kvq_attend import FMT, ints, queries, run, sq  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

# Requests (new tokens, tokens before), heads, key-value heads, width, bound of the lengths: one query a request,
# a few, tiles of 128 rows and tiles of 256.
FORMS = {"token": (None, [0, 15, 16, 70, 149], 4, 1, 64, 0), "few": ([4] * 5, [0, 14, 29, 60, 130], 4, 1, 64, 0),
         "tiles": ([150, 33, 70, 0], [0, 31, 90, 20], 4, 1, 64, 0), "tiles256": ([40, 0, 64, 56], [0, 5, 70, 44], 4, 1, 128, 4400),
         "splits": ([33, 40], [2100, 1500], 4, 1, 64, 0)}


def shape(form):
    new, ctx, H, Hkv, d, most = FORMS[form]
    lens = [a + b for a, b in zip(ctx, new or [1] * len(ctx))]
    cu = [0] + np.cumsum(new or [1] * len(ctx)).tolist()
    return new, ctx, lens, cu, H, Hkv, d, most or max(lens)


def held_scales(c, table, lens, which, of):
    """Scales `of(block of its request)` for keys (0) or values (1)."""
    for r, n in enumerate(lens):
        for i in range(-(-n // 16)):
            c.scales[table[r, 16 * i // c.P], :, 16 * i % c.P // 16, which] = of(i)


def reaches(table, P, most):
    """The table with room for `most` positions: pages that do not exist."""
    more = max(0, -(-most // P) - table.shape[1])
    return np.concatenate([table, np.full((table.shape[0], more), -1, table.dtype)], 1)


def compare(o, lse, w, lim):
    assert torch.isfinite(o).all()
    off = (o - w[0]).abs()
    assert (off <= lim[0]).all(), float((off / lim[0].clamp(min=1e-300)).max())
    off = (lse - w[1]).abs()
    assert (off <= lim[1]).all(), float((off / lim[1]).max())


def check(sq, c, q, table, form, dtype, window=0):
    new, _, lens, cu, _, _, d, most = shape(form)
    o, lse = run(sq, c, q, reaches(table, c.P, most), lens, new, window=window, most=most)
    w = ref.attention(c, q, table, lens, cu, d ** -0.5, window)
    compare(o, lse, w, kw.limits(w, kw.floors(c, q, table, lens, cu, d ** -0.5, window), dtype))


# ---------------------------------------------------------------- blocks of zeros

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
def test_blocks_of_zeros_beside_large_values(sq, fmt, dtype, form):
    """Padding and the like: blocks whose values are all zero, written by sq_kvq_append, before, after and among
    blocks of large ones.  Their tokens count in the softmax as all others."""
    new, ctx, lens, cu, H, Hkv, d, _ = shape(form)
    g = torch.Generator().manual_seed(3)
    table, pages = ref.tables(lens, 16, g)
    at = [0] + np.cumsum(lens).tolist()
    block = torch.cat([torch.arange(n) // 16 for n in lens])
    q = queries(4, cu[-1], H, d, dtype)
    for large, zero in ((1e3, (0, 2, 3, 7)), (1e9, (1, 2, 3, 8)), (1e13, (0, 1, 3, 4, 5)), (1e30, (0, 4, 5, 6, 7)),
                        (1e30, (1, 3, 5, 7, 9))):
        k = 0.1 * torch.randn(at[-1], Hkv, d, generator=g)
        v = large * torch.randn(at[-1], Hkv, d, generator=g)
        v[torch.isin(block, torch.tensor(zero))] = 0.0
        c = ref.Cache(pages, Hkv, 16, d, fmt)
        dev = c.gpu(sq)
        sq.sq_kvq_append(dev, k.cuda(), v.cuda(), ints([0] * len(lens)), ints(at), torch.from_numpy(table).cuda())
        c.append(k, v, [0] * len(lens), at, table)
        c.same(dev)
        check(sq, c, q, table, form, dtype)


# ---------------------------------------------------------------- scores of any size

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("power", [10, 17, 25, 28, 99])
def test_large_scores_that_are_equal(sq, fmt, dtype, form, power):
    """Equal keys have equal weights, whatever the scores are; where some keys' scores are larger, those have."""
    new, _, lens, cu, H, Hkv, d, most = shape(form)
    c, table = ref.filled(lens, 16, Hkv, d, fmt, power)
    key = torch.randint(1, 100, (d,), generator=torch.Generator().manual_seed(1))
    sharp = ref.Cache.__new__(ref.Cache)
    sharp.__dict__.update(c.__dict__)
    c.k[:] = (128 + key if fmt == "int8" else key.float().to(torch.float8_e4m3fn).view(torch.uint8)).to(torch.uint8)
    sharp.k = c.k.clone()
    one = 128 + 120 if fmt == "int8" else 0x70  # 128 as e4m3
    for r, n in enumerate(lens):
        for x in range(0, n, 37):
            sharp.k[table[r, x // 16], :, x % 16] = one
    held_scales(c, table, lens, 0, lambda i: 0.01)
    for cc, q in ((c, queries(2, cu[-1], H, d, dtype)), (sharp, queries(2, cu[-1], H, d, dtype).abs() + 0.5)):
        scale = 2.0 ** power / 64
        o, lse = run(sq, cc, q, reaches(table, 16, most), lens, new, scale=scale, most=most)
        # Weights are equal, or zero (some 100 nats below the others and more, all scores of one key are one
        # number): 64 bits have them at a smaller scale, and what scores are rounded by does not enter o.
        small = 0.0 if cc is c else min(scale, 2.0 ** 10 / 64)
        floor = kw.floors(cc, q, table, lens, cu, small)
        w = list(ref.attention(cc, q, table, lens, cu, small, 0))
        w[3] = torch.zeros_like(w[3])
        lim_o, _ = kw.limits(w, floor, dtype)
        w[1], _, size = ref.attention(cc, q, table, lens, cu, scale, 0)[1:4]
        w[3] = size
        compare(o, lse, w, (lim_o, kw.limits(w, floor, dtype)[1]))


# ---------------------------------------------------------------- value scales of tokens that a row does not see

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("step,window", [(3, 0), (10, 0), (20, 0), (-10, 20), (-20, 40)])
def test_value_scales_of_tokens_not_seen(sq, fmt, dtype, form, step, window):
    """Value scales that rise from block to block, by 2^3 to 2^20 (four blocks, then from the start), and fall in
    front of a window: a row's weights have their bits beside what later rows see."""
    new, _, lens, cu, H, Hkv, d, _ = shape(form)
    c, table = ref.filled(lens, 16, Hkv, d, fmt, 31)
    held_scales(c, table, lens, 0, lambda i: 1 / 64)
    held_scales(c, table, lens, 1, lambda i: 1.3 * 2.0 ** (step * (i % 4) - 2))
    check(sq, c, queries(5, cu[-1], H, d, dtype), table, form, dtype, window)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
def test_large_values_of_small_weight(sq, fmt, dtype, form):
    """Tokens of value scales 2^40 and weights near 2^-60 beside others of 2^-20 and 1."""
    new, _, lens, cu, H, Hkv, d, _ = shape(form)
    c, table = ref.filled(lens, 16, Hkv, d, fmt, 33)
    held_scales(c, table, lens, 1, lambda i: 2.0 ** 40 if i % 3 == 1 else 0.7 * 2.0 ** -20)
    # keys of one code: + in most blocks, - where values are large; queries of one sign
    for r, n in enumerate(lens):
        for x in range(n):
            far = x // 16 % 3 == 1
            c.k[table[r, x // 16], :, x % 16] = (128 - 64 if far else 128 + 64) if fmt == "int8" else (0xe8 if far else 0x68)
    held_scales(c, table, lens, 0, lambda i: 1 / 64)
    q = (1 + 0.01 * queries(5, cu[-1], H, d, dtype).float().abs()) * (20.6 / d ** 0.5)  # scores of +-20.6: e^41 is 2^60
    check(sq, c, q.to(ref.DT[dtype]), table, form, dtype)


# ---------------------------------------------------------------- the bits of fp32 calls

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("form", ["token", "few", "tiles"])
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("size", [0.5, 16.0])
def test_full_precision_of_f32(sq, fmt, form, d, size):
    """Few tokens, and queries of one value that is not zero: 22 bits of query and weight are all there."""
    new = {"token": None, "few": [3, 2, 3, 1], "tiles": [5, 5, 3, 6]}[form]
    lens = {"token": [2, 3, 5, 2, 3], "few": [3, 3, 5, 2], "tiles": [5, 6, 3, 7]}[form]
    cu = [0] + np.cumsum(new or [1] * len(lens)).tolist()
    H = 16 if form == "tiles" else 4
    c, table = ref.filled(lens, 16, 1, d, fmt, d)
    g = torch.Generator().manual_seed(d)
    q = torch.zeros(cu[-1], H, d)
    at = torch.randint(0, d, (cu[-1], H, 1), generator=g)
    top = 64 * (127 if fmt == "int8" else 120) ** -1.0
    q.scatter_(2, at, size * top * (0.5 + 0.5 * torch.rand(cu[-1], H, 1, generator=g)))
    o, _ = run(sq, c, q, table, lens, new, scale=1.0)
    w = ref.attention(c, q, table, lens, cu, 1.0, 0)
    lim = kw.exact_limits(w, kw.floors(c, q, table, lens, cu, 1.0), max(lens))
    off = (o - w[0]).abs()
    assert (off <= lim).all(), float((off / lim).max())
