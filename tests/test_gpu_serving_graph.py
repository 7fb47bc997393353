"""The serving operators captured together: a graph of prompts (tables, the
prompt form, append) and of a token's attention, replayed for other lengths with
eager work between, against the same calls made eagerly."""
import pytest
import torch

from test_gpu_prefill import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("n,most", [(2, 2600), (3, 90)])
def test_prompts_and_attention(sq, rule, n, most):
    """2 x 2,600 tokens of plain decay go through segments; the token count is the
    graph's capacity, the lengths are the device's."""
    H, kv, qh, d, P, N = 2, 2, 4, 128, 16, n * most
    x = make(5 + n, [N], H, H, d, d, "bf16", init=False)
    q, k, v, al, be = (x[m].cuda() for m in ("q", "k", "v", "alpha", "beta"))
    i32 = dict(dtype=torch.int32, device="cuda")
    cols = -(-most // P)
    ak, av = torch.randn(N, kv, d, device="cuda").bfloat16(), torch.randn(N, kv, d, device="cuda").bfloat16()
    aq = torch.randn(n, qh, d, device="cuda").bfloat16()
    ctx, new, free = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.randperm(n * cols, device="cuda").to(torch.int32)
    nb = sq.sq_prefill_workspace(n, N, H, d, d, torch.bfloat16, rule)
    assert (nb > 0) == (rule == 1 and most == 2600)

    class Side:
        def __init__(self):
            self.cache = sq.SqKvCache(torch.zeros(n * cols, kv, P, d, device="cuda").bfloat16(),
                                      torch.zeros(n * cols, kv, d, P, device="cuda").bfloat16())
            self.table, self.seq = torch.full((n, cols), -1, **i32), torch.zeros(n, **i32)
            self.cu, self.cp, self.res = (torch.zeros(m, **i32) for m in (n + 1, n + 1, 1))
            self.slots = torch.zeros(N, dtype=torch.int64, device="cuda")
            self.o, self.S = torch.zeros_like(v), torch.zeros(n, H, d, d, device="cuda")
            self.ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")
            self.ao, self.lse = torch.zeros_like(aq), torch.zeros(n, qh, device="cuda")
            self.aws = torch.empty(max(256, sq.sq_paged_attention_workspace(self.cache, n, qh, most)),
                                   dtype=torch.uint8, device="cuda")

        def call(self):
            sq.sq_block_tables(ctx, new, P, free, self.table, self.seq, self.cu, self.cp, self.slots, self.res)
            sq.sq_prefill(q, k, v, al, be, self.cu, self.o, S=self.S, rule=rule, workspace=self.ws)
            sq.sq_kv_append(self.cache, ak, av, self.slots)
            sq.sq_paged_attention(self.cache, aq, self.table, self.seq, most, self.ao, self.aws, lse=self.lse)

        def out(self):
            used = int(self.cu[-1])  # tokens after the last one are nobody's
            return [t.clone() for t in (self.table, self.seq, self.cu, self.cp, self.slots, self.res, self.o[:used],
                                        self.S, self.ao, self.lse, self.cache.k, self.cache.v)]

    a, b = Side(), Side()
    for side in (a, b):  # once outside a capture
        side.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call()
    for lens in ([most] * n, [1, most - 7] + [0] * (n - 2), [0] * n, [most // 2, 65] + [64] * (n - 2)):
        new.copy_(torch.tensor(lens, **i32))
        graph.replay()
        b.call()
        torch.cuda.synchronize()
        for x1, x2 in zip(a.out(), b.out()):
            assert torch.equal(x1, x2)
        assert int(a.res) == 0 and a.cu.tolist()[-1] == sum(lens)
        v.mul_(0.5)
