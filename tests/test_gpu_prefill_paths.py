"""sq_prefill on its less travelled paths: the token-by-token kernel of many
columns, and how exact a state is.

Tolerances as in test_gpu_prefill, unless said."""
import numpy as np
import pytest
import torch

import serve_reference as ref
from test_gpu_prefill import check, make, run


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


# ---------------------------------------------------------------- token by token, 4 lanes a column
#
# taken above 12,288 columns (sequences x heads x d_v)

@pytest.mark.gpu
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,H", [(64, 64, 52), (60, 200, 16), (4, 256, 13), (128, 136, 24), (100, 128, 26),
                                     (256, 64, 50), (132, 200, 16)])
def test_many_columns(sq, rule, dtype, dk, dv, H):
    lens = [0, 1, 17, 33]
    assert len(lens) * H * dv > 12288
    check(sq, make(dk + dv, lens, H, H // 2 if H % 2 == 0 else H, dk, dv, dtype), rule, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("H", [96, 97])
def test_on_both_sides_of_many_columns(sq, rule, H):
    for dtype, lens in (("f32", [35]), ("bf16", [12])):
        check(sq, make(H, lens, H, H, 128, 128, dtype), rule, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("init", [False, True])
def test_a_few_tokens_of_many_sequences(sq, rule, init):
    """12 tokens a sequence on average and no more: one by one, also in bfloat16
    at d = 128 and for the one long sequence among them."""
    lens = [12, 0, 1, 11, 3, 70, 2, 9, 5, 0, 7, 24]
    assert sum(lens) == 12 * len(lens)
    check(sq, make(53, lens, 12, 4, 128, 128, "bf16", init), rule, "bf16")


# ---------------------------------------------------------------- how exact a state is
#
# Everything that feeds a state is fp32 or better: per 64 tokens a state element
# takes some fourteen fp32 roundings (a scaling, six products of 64 keys, and
# what the writes bring from a dozen more), at random, while what the tokens
# before left decays; a gate's product is off by a unit or two, over the twenty
# chunks or so that the slowest head remembers.  Their squares add up to about
# 12 units of 2^-24 of the state's size (root of the sum of squares); 32 are
# allowed.  Values cut to two bfloat16 planes (16 bits, towards zero) would be
# off by 100 to 200: the second test.

BAR = 32 * 2.0 ** -24


def distance(got, want):
    """||got - want|| / ||want|| of every state."""
    d = np.sqrt(((got - want) ** 2).sum((-1, -2)))
    return d / np.sqrt((want ** 2).sum((-1, -2)))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype,lens,H", [("bf16", [64, 500, 1027], 3), ("bf16", [200], 130), ("bf16", [4000], 2),
                                          ("f32", [64, 300], 3)])
def test_states_are_fp32(sq, rule, dtype, lens, H):
    x = make(71, lens, H, H, 128, 128, dtype, init=False)
    _, S = run(sq, x, rule)
    _, want = ref.prefill(x["q"].float(), x["k"].float(), x["v"].float(), x["alpha"], x["beta"], x["cu"], None, rule == 0)
    assert (distance(S, want) <= BAR).all(), distance(S, want).max() * 2 ** 24


def cut(x, bits):
    """x with `bits` bits of mantissa, cut towards zero."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, bits)), e - bits)


def test_states_of_fewer_bits_would_not_pass():
    x = make(73, [300], 2, 2, 128, 128, "bf16", init=False)
    args = [x[m].float().numpy().astype(np.float64) for m in ("q", "k", "v", "alpha", "beta")]
    _, k, v, al, be = args
    S, C = np.zeros((2, 128, 128)), np.zeros((2, 128, 128))
    for t in range(300):
        for R, bits in ((S, 60), (C, 16)):
            w = be[t][:, None] * (v[t] - al[t][:, None] * np.einsum("hi,hij->hj", k[t], R))
            R *= al[t][:, None, None]
            R += k[t][:, :, None] * cut(w, bits)[:, None, :]
    _, want = ref.prefill(*(torch.from_numpy(a) for a in args), x["cu"], None, True)
    assert (distance(S, want) <= 1e-12).all()
    assert (distance(C, want) > BAR).all(), distance(C, want) * 2 ** 24
