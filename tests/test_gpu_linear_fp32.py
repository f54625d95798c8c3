"""fp32 results of moe_linear: the activations far from zero."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe

from test_gpu_linear import workspace

pytestmark = pytest.mark.gpu


def through(values, act, T, dtype):
    """act(values) of the call: x picks one column of w, so the sums are exact."""
    N = values.numel()
    w = torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 3] = values
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 1.0
    out = torch.empty(T, N, dtype=dtype, device="cuda")
    moe.moe_linear(x, w, out, workspace(T, N, 8), activation=act)
    return out


@pytest.mark.parametrize("T", [3, 70, 300])
def test_silu_far_from_zero(T):
    """v / (1 + exp(-v)): exp within 2 ulps (CUDA's bound of expf), the sum and the
    quotient within half an ulp each, an ulp being at most 2^-23 of its value: 3 x 2^-23.
    Down to -80, where exp(80) is still finite."""
    v = torch.cat([torch.linspace(-80, 80, 4097), torch.linspace(-2, 2, 513)]).to(torch.bfloat16).cuda()
    got = through(v, "silu", T, torch.float32).double()
    want = v.double() * torch.sigmoid(v.double())
    assert ((got - want).abs() <= 3 * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("T", [3, 300])
def test_silu_bf16_is_the_rounded_value(T):
    """The approximate exponential's 2 + 1.17 |v| ulps and the reciprocal's one, under the rounding."""
    v = torch.linspace(-80, 80, 4097).to(torch.bfloat16).cuda()
    got = through(v, "silu", T, torch.bfloat16).double()
    want = v.double() * torch.sigmoid(v.double())
    assert ((got - want).abs() <= (2.0 ** -8 + (2 + 1.173 * v.double().abs() + 2) * 2.0 ** -23) * want.abs()).all()


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_activations_of_huge_values(T, dtype):
    v = torch.tensor([-3.0e38, -1e4, -200.0, 200.0, 1e4, 3.0e38, 0.0, float("nan")]).to(torch.bfloat16).cuda()
    for act in ("silu", "gelu", "relu"):
        got = through(v, act, T, dtype)
        assert (got[:, :3] == 0).all() and (got[:, 3:6] == v[3:6].to(dtype)).all() and (got[:, 6] == 0).all()
        assert got[:, 7].isnan().all()
