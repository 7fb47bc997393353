"""sq_prefill where values and outputs lie past 2^31 elements: the last sequence of
a long batch, some of its heads, against the recurrence in 64 bits.

Tolerances as in test_gpu_prefill."""
import numpy as np
import pytest
import torch

import serve_reference as ref
from test_gpu_prefill import DT, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(sq, dtype, rule):
    H, d, lens = 1024, 128, [16900, 70]
    N = sum(lens)
    assert lens[0] * H * d > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(N, 1, d), dim=-1).to(DT[dtype]) for _ in range(2))
    v = torch.empty(N, H, d, dtype=DT[dtype], device="cuda").normal_(generator=g)
    alpha, beta = (0.5 + 0.5 * torch.rand(N, H, generator=g, device="cuda") for _ in range(2))
    cu = np.array([0, lens[0], N], np.int32)
    o, S = torch.empty_like(v), torch.empty(2, H, d, d, device="cuda")
    sq.sq_prefill(q, k, v, alpha, beta, torch.from_numpy(cu).cuda(), o, S=S, rule=rule)
    torch.cuda.synchronize()
    heads = [0, 1, 500, H - 1]
    part = slice(lens[0], N)
    cut = [x[part].float().cpu() for x in (q, k)] + [x[part][:, heads].float().cpu() for x in (v, alpha, beta)]
    wo, wS = ref.prefill(*cut, [0, lens[1]], None, rule == 0)
    close(o[part][:, heads].float().cpu().numpy().astype(np.float64), wo, lens[1], d, dtype == "bf16", "o")
    close(S[1][heads].cpu().numpy().astype(np.float64), wS[0], lens[1], d, False, "S")
