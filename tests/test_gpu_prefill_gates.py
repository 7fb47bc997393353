"""sq_prefill with gates of zero, or next to it, again and again inside 64 tokens:
the running sums of their logarithms are then in the thousands, and what lies
between two of them still has to be weighed exactly.

Tolerances as in test_gpu_prefill."""
import pytest
import torch

from test_gpu_prefill import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("low", [0.0, 1e-44, 1e-30])
@pytest.mark.parametrize("every", [2, 3, 5, 16])
def test_forgetting_again_and_again(sq, rule, low, every):
    x = make(81 + every, [200, 64], 4, 4, 128, 128, "bf16")
    x["alpha"][every - 1::every] = low
    x["alpha"][:, 1] = torch.where(x["alpha"][:, 1] == low, low, 1.0)
    check(sq, x, rule, "bf16")


@pytest.mark.parametrize("rule", [0, 1])
def test_forgetting_in_segments(sq, rule):
    """Long enough for the plain decay's segments."""
    x = make(91, [5000], 2, 2, 128, 128, "bf16")
    x["alpha"][1::2, 0] = 0.0
    x["alpha"][6::7, 1] = 0.0
    check(sq, x, rule, "bf16")


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("low", [0.0, 1e-30])
@pytest.mark.parametrize("every", [2, 3, 5, 16])
def test_forgetting_again_and_again_with_one_key(sq, rule, low, every):
    """All queries and keys alike: an output is the weighted sum of the last few
    writes, and small where they cancel."""
    x = make(81 + every, [200, 64], 4, 4, 128, 128, "bf16", init=False, keys="same")
    x["q"] = x["k"].clone()
    x["alpha"][:] = 0.8 + 0.2 * torch.rand(x["alpha"].shape, generator=torch.Generator().manual_seed(every))
    x["alpha"][every - 1::every] = low
    x["beta"][:] = 0.5
    check(sq, x, rule, "bf16")
