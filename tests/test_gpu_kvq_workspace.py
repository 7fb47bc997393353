"""The workspace of sq_kvq_attention: the least that a call accepts is all that it writes, and the
size that callers are told, or that of a larger call, gives the same bits."""
import numpy as np
import pytest
import torch

import kvq_reference as ref
from test_gpu_kvq_attend import ints, queries, sq  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

# new tokens (None: one a request), tokens before, heads, key-value heads, width, window
CALLS = [(None, [3000, 5, 700], 4, 1, 64, 0), (None, [9000], 17, 1, 32, 0), ([1, 2, 3, 33], [4000, 2500, 90, 2200], 4, 1, 64, 0),
         ([33], [9000], 8, 2, 128, 0), ([40, 1, 0, 70], [5000, 6000, 40, 100], 3, 1, 96, 2500), ([3, 1], [4000, 3000], 5, 1, 256, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("call", range(len(CALLS)))
def test_workspace(sq, dtype, call):
    new, ctx, H, Hkv, d, window = CALLS[call]
    lens = [a + b for a, b in zip(ctx, new or [1] * len(ctx))]
    c, t = ref.filled(lens, 16, Hkv, d, "int8", call)
    dev, table = c.gpu(sq), torch.from_numpy(t).cuda()
    q = queries(call, sum(new or [1] * len(ctx)), H, d, dtype).cuda()
    cu = None if new is None else ints([0] + np.cumsum(new).tolist())
    n, most = len(lens), max(lens)
    told = sq.sq_kvq_attention_workspace(dev, n, q.shape[0], H, most)
    larger = sq.sq_kvq_attention_workspace(dev, n + 3, q.shape[0] + 50, H, most + 3000)
    buf = torch.empty(larger + 4096, dtype=torch.uint8, device="cuda")

    def outputs(size):
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        buf.fill_(0xa5)
        sq.sq_kvq_attention(dev, q, table, ints(lens), most, o, buf[:size], cu_q=cu, window=window, lse=lse)
        torch.cuda.synchronize()
        assert (buf[size:] == 0xa5).all()
        return o, lse

    refused, least = 0, told
    with pytest.raises(sq.SqError):
        outputs(0)
    while least - refused > 16:
        size = (least + refused) // 32 * 16
        size = size if refused < size < least else refused + 16
        try:
            outputs(size)
            least = size
        except sq.SqError:
            refused = size
    o, lse = outputs(least)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    for size in (told, larger):
        o2, lse2 = outputs(size)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
