"""sq_block_tables with lengths far past the table: reported, in the time of the
rows that exist, not of the pages asked for."""
import time

import numpy as np
import pytest
import torch

from test_gpu_paged import check_tables, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


@pytest.mark.parametrize("n", [3, 40, 2100])
def test_rows_overrun_by_some(sq, n):
    """Rows that overrun by a few pages, by many workgroups' worth, and not at all."""
    rng = np.random.default_rng(n)
    ctx = [int(x) for x in rng.integers(0, 200, n)]
    new = [int(x) for x in rng.choice([0, 1, 17, 90, 700, 20000, 90000], n, p=[.2, .2, .2, .2, .185, .01, .005])]
    if n == 3:
        new = [90000, 3, 700]
    table = np.arange(n * 12).reshape(n, 12)
    check_tables(sq, ctx, new, 16, [int(x) for x in rng.permutation(5000)], table, 4000)


@pytest.mark.parametrize("n", [64, 2500])
def test_the_largest_lengths(sq, n):
    """2^31 - 1 new tokens each: the sums stop at 2^31 - 1, the call soon after
    it began (walking all pages would take seconds)."""
    top = 2 ** 31 - 1
    ctx, new = [0, 5] + [0] * (n - 2), [3, top - 5] + [top] * (n - 2)
    args = (sq, ctx, new, 16, [7, 9, 11], np.full((n, 4), -5), 100)
    tables(*args)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    t, seq, cn, cp, slots, result = tables(*args)
    assert time.perf_counter() - t0 < 0.5
    assert result == 2 | 4 | 8 and list(seq) == [c + m for c, m in zip(ctx, new)]
    assert list(cn[:4]) == [0, 3, top - 2, top] and list(cp[:3]) == [0, 1, 2 ** 27] and cn[-1] == cp[-1] == top
    assert list(t[0]) == [7, -5, -5, -5] and list(t[1]) == [-5, 9, 11, -1]
    # request 1 holds a page that its row does not list (-5): its tokens there have no slot
    want = [7 * 16 + x for x in range(3)] + [-1] * 11 + [9 * 16 + x for x in range(16)] + [11 * 16 + x for x in range(16)]
    assert list(slots) == want + [-1] * (100 - len(want))
