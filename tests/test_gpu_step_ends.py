"""Router losses of logits at the ends of their type."""
import pytest
import torch

from fine_grained_mixture_top_amd import ops

import step_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(1, 4), (1, 5), (1, 700), (2, 64), (3, 1024)])
def test_balance_gradient_of_rows_at_their_types_ends(T, E, dtype):
    """A token masked by the type's lowest value throughout (one expert by -inf), beside ordinary ones: 2 lse / n is past
    fp32's range, times a probability it is not."""
    z = torch.randn(T, E, generator=torch.Generator("cuda").manual_seed(E), device="cuda").to(dtype)
    z[0] = torch.finfo(dtype).min
    z[0, 1] = float("-inf")
    idx = torch.arange(T * 2, device="cuda", dtype=torch.int32).view(T, 2) % E
    b = ops.Balance(T, 2, E)
    ops.moe_balance(b, z, idx)
    ref = R.balance_ref(z, idx)
    assert float(b.loss[1]) == float("inf")  # lse^2
    R.within(b.lse, ref["lse"], R.lse_bound(ref["lse"]), "lse")
    d_loss, dz = torch.tensor([0.5, float(T)], device="cuda"), torch.empty_like(z)
    ops.moe_balance_bwd(b, z, d_loss, dz)
    want, bound = R.balance_bwd_ref(z, idx, ref, d_loss)
    assert bool(torch.isfinite(want).all()) and float(want[0].abs().max()) > 1e35
    R.within(dz, want, bound + R.HALF[dtype] * want.abs() + 1e-38, "dz")
    assert float(dz[0, 1]) == 0.0
