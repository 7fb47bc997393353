"""sq_prefill with cu_seqlens that lie outside the tokens, fall, or reach the top
of their type: the outputs are undefined, but nothing outside them is touched."""
import pytest
import torch

from test_gpu_prefill import DT, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


GUARD = 8192  # bytes around each output


def guarded(nbytes):
    return torch.full((GUARD + nbytes + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")


def inside(buf, dtype, shape):
    return buf[GUARD:len(buf) - GUARD].view(dtype).view(shape)


def untouched(*bufs):
    return all((b[:GUARD] == 0xa5).all() and (b[len(b) - GUARD:] == 0xa5).all() for b in bufs)


TOP = 2 ** 31 - 1
OFFSETS = [lambda N: [0, N // 2, 10 ** 6], lambda N: [-9, N // 2, N], lambda N: [0, N - 5, 30], lambda N: [N, 0, 0],
           lambda N: [N - 1, 0, N], lambda N: [10 ** 9, 10 ** 9, 10 ** 9], lambda N: [0, TOP, TOP],
           lambda N: [TOP, TOP, TOP], lambda N: [TOP - 3, TOP - 1, TOP], lambda N: [-2 ** 31, N, -2 ** 31],
           lambda N: [-1, TOP, 0]]


@pytest.mark.parametrize("at", range(len(OFFSETS)))
@pytest.mark.parametrize("N,dtype,rule", [(150, "bf16", 0), (150, "bf16", 1), (5200, "bf16", 1), (150, "f32", 0),
                                          (150, "f32", 1)])
def test_nothing_is_written_around_the_outputs(sq, at, N, dtype, rule):
    """Whole walks, segments (5,200 tokens of plain decay) and token by token."""
    n, H, d = 2, 2, 128
    x = make(61, [N // 2, N - N // 2], H, H, d, d, dtype)
    q, k, v, al, be, S0 = (x[m].cuda() for m in ("q", "k", "v", "alpha", "beta", "S0"))
    nb = sq.sq_prefill_workspace(n, N, H, d, d, DT[dtype], rule)
    assert (nb > 0) == (N == 5200)
    ob, sb, wb = guarded(N * H * d * q.element_size()), guarded(n * H * d * d * 4), guarded(nb)
    o, S = inside(ob, q.dtype, (N, H, d)), inside(sb, torch.float32, (n, H, d, d))
    cu = torch.tensor(OFFSETS[at](N), dtype=torch.int32, device="cuda")
    sq.sq_prefill(q, k, v, al, be, cu, o, S=S, S0=S0, rule=rule, workspace=wb[GUARD:GUARD + nb] if nb else None)
    torch.cuda.synchronize()
    assert untouched(ob, sb, wb)
