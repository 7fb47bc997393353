"""How sq_paged_attention cuts long contexts: splits that a table's row really
has room for, the workspace they need, the largest splits.

Tolerances as in test_gpu_paged."""
import numpy as np
import pytest
import torch

from test_gpu_paged import cache, check_attend, ints, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def wide(t, cols):
    """The same table with rows of `cols` entries."""
    return np.concatenate([t, np.full((t.shape[0], cols - t.shape[1]), -1, np.int32)], 1)


GUARD = 4096


@pytest.mark.parametrize("H,Hkv", [(6, 3), (40, 1)])
@pytest.mark.parametrize("n,most", [(1, 20000), (7, 5000), (90, 3001), (700, 130), (700, 530)])
def test_a_workspace_serves_every_smaller_call(sq, H, Hkv, n, most):
    """Made for (n, max_len), it is enough for fewer requests, shorter ones and
    any window; nothing is written past its end."""
    c = sq.SqKvCache(torch.zeros(4, Hkv, 16, 64, device="cuda"), torch.zeros(4, Hkv, 64, 16, device="cuda"))
    room = sq.sq_paged_attention_workspace(c, n, H, most)
    buf = torch.full((room + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")
    refused = 0
    for m in {1, n // 2 + 1, n}:
        q = torch.zeros(m, H, 64, device="cuda")
        o = torch.empty_like(q)
        for ln in sorted({1, 100, 129, 1000, 1100, most // 3, most - 1, most}):
            if ln > most:
                continue
            table = torch.zeros(m, -(-ln // 16), dtype=torch.int32, device="cuda")
            lens = ints([ln] * m)
            for w in (0, 1, 500, ln):
                sq.sq_paged_attention(c, q, table, lens, ln, o, buf[:room], window=w)
                try:
                    sq.sq_paged_attention(c, q, table, lens, ln, o, window=w)
                except sq.SqError as e:
                    assert e.status == sq.SQ_ERR_INVALID
                    refused += 1
    torch.cuda.synchronize()
    assert (buf[room:] == 0xa5).all()
    assert refused > 0 or most <= 256  # most of these calls do split


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("f32", 128)])
def test_a_loose_max_len_splits_otherwise(sq, dtype, P):
    """Rows with room for 60,000 tokens that hold a third of it at most."""
    lens = [20011, 3, 0, 9000]
    k, v, t = cache(P, lens, P, 1, 128, dtype)
    q = queries(3, 4, 3, 128, dtype)
    c = sq.SqKvCache(k.cuda(), v.cuda())
    few, many = (sq.sq_paged_attention_workspace(c, 4, 3, x) for x in (20011, 60000))
    assert many > few
    check_attend(sq, k, v, wide(t, -(-60000 // P)), lens, q, most=60000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 128])
def test_the_largest_splits(sq, dtype, n):
    """Rows of 262,144 tokens: 128 (request, head) pairs take splits of 8,192
    tokens, twice as many would take longer ones and are held to the same.
    A split's page ids (512 of 16 tokens) are then more than a workgroup's threads."""
    lens = [int(x) for x in np.random.default_rng(n).integers(0, 40, n)]
    lens[1], lens[5], lens[n - 1] = 20000, 8193, 8192
    k, v, t = cache(n, lens, 16, 2, 32, dtype, fill=float("nan"))
    t[1, 300], t[1, 1000], t[5, 511] = -1, 2 ** 31 - 1, -7  # also among the ids past the first 256
    check_attend(sq, k, v, wide(t, 16384), lens, queries(n, n, 4, 32, dtype), most=262144)


def test_the_largest_splits_of_a_window(sq):
    """A window longer than a split of 8,192 tokens, that starts inside a page."""
    n, window = 64, 262144
    lens = [i % 5 for i in range(n)]
    lens[7] = window + 77
    k, v, t = cache(3, lens, 16, 2, 32, "bf16")
    check_attend(sq, k, v, t, lens, queries(4, n, 2, 32, "bf16"), window=window, most=2 ** 20)
