"""Prompts of ``hybrid`` for requests that already hold tokens, and tokens of
requests that hold none."""
import numpy as np
import pytest
import torch

import serve_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from quantized_recurrent_state_gated_amd import hybrid as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("rule", [0, 1])
def test_further_prompts_go_on_from_the_states(H, rule):
    n, heads, parts = 3, 2, ([70, 1, 33], [5, 40, 0], [0, 30, 21])
    g = gen(7)
    m = H.HybridLayers(n, heads, [32] * heads, 4, 2, 16, 160, rule)
    xs = [H.activations(sum(p), heads, 4, 2, g) for p in parts]
    outs = [m.prompts(p, x) for p, x in zip(parts, xs)]
    assert m.ctx.tolist() == [sum(p[r] for p in parts) for r in range(n)]
    at = [np.concatenate([[0], np.cumsum(p)]) for p in parts]
    for r in range(n):
        def mine(key):
            return torch.cat([x[key][a[r]:a[r + 1]] for x, a in zip(xs, at)]).float().cpu()
        T = sum(p[r] for p in parts)
        wo, _ = ref.prefill(mine("q"), mine("k"), mine("v"), mine("alpha"), mine("beta"), [0, T], None, rule == 0)
        got = torch.cat([o[a[r]:a[r + 1]] for o, a in zip(outs, at)]).float().cpu().numpy()
        # outputs are rounded to bfloat16; states are fp32 sums over the tokens
        lim = 2.0 ** -8 * np.abs(wo) + (T + 512) * 2.0 ** -24 * np.abs(wo).max()
        assert (np.abs(got - wo) <= lim).all()


@pytest.mark.parametrize("bits", [4, 8, 16, 32])
def test_a_first_token_starts_from_zero(H, bits):
    """Without a prompt: o = beta (q.k) v, whatever the pool's buffer held."""
    junk = torch.full((1 << 26,), 0x5f, dtype=torch.uint8, device="cuda")
    del junk
    m = H.HybridLayers(2, 3, [bits] * 3, 4, 2, 16, 40)
    x = H.activations(2, 3, 4, 2, gen(8))
    o, _ = m.token(x)
    q, k, v, be = (x[n].double() for n in ("q", "k", "v", "beta"))
    want = (be * (q * k).sum(-1))[..., None] * v
    # the bar of the decode step's readout
    assert ((o.double() - want).abs() <= 1e-5 + 1e-3 * want.abs().amax(-1, keepdim=True)).all()
