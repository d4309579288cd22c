"""GELU far from zero: y Phi(y) keeps its relative precision where Phi(y) is small.

Tolerance: an argument y / sqrt 2 that is rounded twice (2^-24 each) moves y Phi(y) by at most (y^2 + 2) 2^-23 of its value,
as do y^2 / 2 rounded twice and its constant in an exponent; beside this a special function has 4 units in the last place
(2^-21), two products 2^-24 each; a bf16 output half its step.  The pre-activations are exact: one product of a row is not
zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("k", [8, 2048])          # one share of the contraction, and several
def test_gelu_tail(rows, k, dtype):
    y = torch.cat([torch.linspace(-12, 0, 800), torch.linspace(0, 12, 200)]).to(torch.bfloat16).cuda()
    x, w = torch.zeros((rows, k), device="cuda", dtype=torch.bfloat16), torch.zeros((1000, k), device="cuda", dtype=torch.bfloat16)
    x[:, 3], w[:, 3] = 1, y
    got = mk.linear(x, w, activation="gelu", out_dtype=dtype).double()
    y = y.double()
    want = y * torch.special.erfc(-y / 2 ** 0.5) / 2
    bound = ((y * y + 2) * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -23 + (2.0 ** -8 if dtype == torch.bfloat16 else 0)) * want.abs() + 1e-37
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max().item()


def test_gelu_of_what_is_not_finite():
    x, w = torch.zeros((5, 8), device="cuda", dtype=torch.bfloat16), torch.zeros((2, 8), device="cuda", dtype=torch.bfloat16)
    w[:, 0] = 1
    x[:, 0] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3e38, -3e38])
    y = mk.linear(x, w, activation="gelu", out_dtype=torch.float32)
    assert (y[0] == float("inf")).all() and y[1:3].isnan().all()          # (-inf times 0, as the formula has it)
    assert (y[3] == x[3, 0].float()).all() and (y[4] == 0).all()
