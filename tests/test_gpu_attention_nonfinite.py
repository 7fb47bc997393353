"""sq_paged_attention where a live query, key or value is not finite, or a score
overflows.  The softmax of such scores has no value: NaN, in the output and in
the log sum, for exactly the heads that meet it.  Zeros with a log sum of -inf
are for requests that have no tokens, whatever the scores of the others are."""
import numpy as np
import pytest
import torch

import serve_reference as ref
from test_gpu_paged import attend, cache, queries

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
LENS = [1, 40, 300, 3000, 0]  # one tile, two, several rounds of four waves, several splits, none


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def only_these_are_nan(got, clean, hit):
    """o, lse of both runs; hit [n][H]: NaN in whole rows there, the clean run's bits elsewhere."""
    (o, l), (wo, wl) = got, clean
    assert np.isnan(o[hit]).all() and np.isnan(l[hit]).all()
    assert np.array_equal(o[~hit], wo[~hit]) and np.array_equal(l[~hit], wl[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 35])
def test_nan_in_a_query(sq, dtype, window):
    k, v, t = cache(41, LENS, 16, 2, 64, dtype)
    q = queries(41, 5, 6, 64, dtype)
    clean = attend(sq, k, v, t, LENS, q, window=window)
    q[:, 1, 9] = NAN
    q[3, 5, 0] = INF  # meets keys of both signs
    hit = np.zeros((5, 6), bool)
    hit[:4, 1] = hit[3, 5] = True  # the last request has no tokens
    only_these_are_nan(attend(sq, k, v, t, LENS, q, window=window), clean, hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [slice(0, 1), slice(299, 300), slice(32, 64), slice(16, 32), slice(0, 300)])
def test_nan_in_keys(sq, dtype, at):
    """One key, the whole tile of one of the four waves, or all of them."""
    k, v, t = cache(43, LENS, 16, 2, 64, dtype)
    q = queries(43, 5, 6, 64, dtype)
    clean = attend(sq, k, v, t, LENS, q)
    for r in (2, 3):
        for x in range(at.start, at.stop):
            k[t[r, x // 16], 1, x % 16, 3] = NAN
    hit = np.zeros((5, 6), bool)
    hit[2:4, 3:] = True
    only_these_are_nan(attend(sq, k, v, t, LENS, q), clean, hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,sign", [(32, -1.0), (64, -1.0), (128, 1.0), (256, -1.0)])
def test_scores_that_overflow(sq, dtype, d, sign):
    """Finite queries and keys whose every product passes the fp32 range."""
    k, v, t = cache(45, LENS, 16, 2, d, dtype)
    q = queries(45, 5, 6, d, dtype)
    for r, n in enumerate(LENS):  # keys of head 0: positive
        for x in range(n):
            k[t[r, x // 16], 0, x % 16] = 1e30
    clean = attend(sq, k, v, t, LENS, q)
    q[:, 2] = sign * 1e30
    hit = np.zeros((5, 6), bool)
    hit[:4, 2] = True
    only_these_are_nan(attend(sq, k, v, t, LENS, q), clean, hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_some_scores_overflow_to_minus_infinity(sq, dtype):
    """They weigh nothing; the others share the sum.  Also where the first tiles
    and splits have none of the others."""
    k, v, t = cache(47, LENS, 16, 1, 64, dtype)
    q = queries(47, 5, 2, 64, dtype)
    q[:, 1] = -1e30
    seen = []
    for r, n in enumerate(LENS):
        live = [x for x in range(n) if x >= n - 1 - n // 10]
        for x in range(n):
            k[t[r, x // 16], 0, x % 16] = 0.0 if x in live else 1e30
        seen.append(live)
    o, l = attend(sq, k, v, t, LENS, q)
    vals = v.float().numpy()
    for r in range(4):
        x = np.array(seen[r])
        rows = vals[t[r, x // 16], 0, :, x % 16].astype(np.float64)
        # equal scores of zero: equal weights, by the bounds of the other tests
        lim = 2.0 ** -14 * np.abs(rows).mean(0) + 2.0 ** -8 * np.abs(rows.mean(0))
        assert (np.abs(o[r, 1] - rows.mean(0)) <= lim).all()
        assert abs(l[r, 1] - np.log(len(x))) <= 2.0 ** -14 + 2.0 ** -18 * (1 + np.log(len(x)))
    assert not o[4].any() and np.isneginf(l[4]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [NAN, INF])
def test_nonfinite_values_stay_in_their_column(sq, dtype, what):
    k, v, t = cache(49, LENS, 16, 2, 64, dtype)
    q = queries(49, 5, 4, 64, dtype)
    o, l = attend(sq, k, v, t, LENS, q)
    v[t[2, 3], 1, 5, 2], v[t[3, 100], 0, 63, 15] = what, what
    o2, l2 = attend(sq, k, v, t, LENS, q)
    hit = np.zeros(o.shape, bool)
    hit[2, 2:, 5] = hit[3, :2, 63] = True
    assert not np.isfinite(o2[hit]).any()
    assert np.array_equal(o2[~hit], o[~hit]) and np.array_equal(l2, l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_requests_whose_pages_are_all_missing_have_no_tokens(sq, dtype):
    lens = [64, 3000, 64]
    k, v, t = cache(51, lens, 16, 1, 64, dtype)
    t[:2] = -1
    q = queries(51, 3, 2, 64, dtype)
    q[0, 0, 0] = NAN  # there is no score that it could reach
    o, l = attend(sq, k, v, t, lens, q)
    assert not o[:2].any() and np.isneginf(l[:2]).all()
    kk, vv = k.float().numpy(), v.float().numpy()
    wo, wl, mag = ref.attention(q[2:].float().numpy(), kk, vv, t[2:], lens[2:], 0.125, 0)
    assert (np.abs(o[2:] - wo) <= 2.0 ** -14 * mag + 2.0 ** -8 * np.abs(wo)).all()
    assert (np.abs(l[2:] - wl) <= 2.0 ** -14 + 2.0 ** -18 * (1 + np.abs(wl))).all()
