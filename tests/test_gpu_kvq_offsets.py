"""Offsets that fall (a caller's mistake) in the 8-bit cache's calls: requests' pages and rows
are found by them, and what lies in front of a table, a query or an output must not be touched."""
import numpy as np
import pytest
import torch

import kvq_reference as ref
from test_gpu_kvq_attend import FMT, ints, queries, sq  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def falling(rng, n, most):
    """Offsets that rise from request to request, but for some in the middle."""
    cu = np.sort(rng.integers(0, most + 1, n + 1))
    at = rng.integers(1, n, max(1, n // 8))
    cu[at] = rng.integers(-50, most + 50, len(at))
    return cu.tolist()


CU = [[0, 100, 160, 5, 160], [160, 0, 160, 0, 160], [0, 160, 0, 0, 160]]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n", [4, 300])
def test_rows(sq, fmt, n):
    """Pages of the requests' own rows may be written, all others hold what they held: those that lie in front
    of the table among them."""
    rng = np.random.default_rng(n)
    H, P, d, cols, N = 2, 16, 64, 12, 160
    own, other = n * cols, 64
    c = ref.Cache(own + other, H, P, d, fmt)
    c.scales[own:] = 0.0  # a call that goes on in such a block raises it
    dev = c.gpu(sq)
    rows = torch.empty(16 + n, cols, dtype=torch.int32)
    rows[:16] = own + torch.randint(0, other, (16, cols), generator=torch.Generator().manual_seed(n)).int()
    rows[16:] = torch.arange(own).view(n, cols).int()
    table = rows.cuda()[16:]
    x = torch.randn(N, H, d, device="cuda")
    ko, vo = (torch.full((N + 8, H, d), 7.0, device="cuda") for _ in range(2))
    for cu in (CU if n == 4 else [falling(rng, n, N) for _ in range(4)]):
        for start in (0, 21):
            ctx = ints([start] * n)
            sq.sq_kvq_append(dev, x, x, ctx, ints(cu), table)
            sq.sq_kvq_load(dev, table, ints(cu), ko[:N], vo[:N], first=ctx)
            torch.cuda.synchronize()
            assert torch.equal(dev.k[own:].cpu(), c.k[own:]) and torch.equal(dev.v[own:].cpu(), c.v[own:])
            assert torch.equal(dev.scales[own:].cpu(), c.scales[own:])
            assert (ko[N:] == 7).all() and (vo[N:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,most", [(4, 300), (4, 3000), (100, 300), (100, 3000), (300, 300)])
def test_queries(sq, dtype, n, most):
    """Many requests are found by a search, few by a count; splits are joined by a search too.  Guards
    before and behind the outputs stay."""
    rng = np.random.default_rng(n + most)
    H, d, N = 8, 64, 700
    lens = [int(v) for v in rng.integers(1, 100, n)]
    lens[:3] = [most, most - 1, most // 2]
    c, t = ref.filled(lens, 64, 1, d, "int8", n)
    dev, table = c.gpu(sq), torch.from_numpy(t).cuda()
    q = queries(3, N, H, d, dtype).cuda()
    o = torch.full((N + 400, H, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((N + 400, H), 7.0, device="cuda")
    nb = sq.sq_kvq_attention_workspace(dev, n, N, H, most)
    ws = torch.zeros(max(nb, 1), dtype=torch.uint8, device="cuda")
    for cu in [falling(rng, n, N) for _ in range(6)]:
        sq.sq_kvq_attention(dev, q, table, ints(lens), most, o[200:-200], ws, cu_q=ints(cu), lse=lse[200:-200])
        torch.cuda.synchronize()
        for g in (o[:200], o[-200:], lse[:200], lse[-200:]):
            assert (g == 7).all()
