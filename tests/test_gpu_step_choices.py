"""Balance losses of tokens with more choices than experts (an id may come more than once), in the form of
one workgroup and in that of many."""
import pytest
import torch

from fine_grained_mixture_top_amd import ops

import step_ref as R
from test_gpu_step_ops import check_balance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K", [(16384, 1, 1024), (16, 8, 1024), (17, 8, 1024), (512, 32, 33), (5000, 3, 200)])
def test_balance_of_many_choices(T, E, K):
    g = torch.Generator("cuda").manual_seed(T + K)
    z = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.randint(-1, E + 1, (T, K), generator=g, device="cuda", dtype=torch.int32)
    b = ops.Balance(T, K, E)
    b.ws.fill_(255)
    ops.moe_balance(b, z, idx)
    ref = check_balance(b, z, idx, None)
    d_loss, dz = torch.tensor([0.7, 0.3], device="cuda"), torch.empty_like(z)
    ops.moe_balance_bwd(b, z, d_loss, dz)
    want, bound = R.balance_bwd_ref(z, idx, ref, d_loss)
    R.within(dz, want, bound + R.HALF[z.dtype] * want.abs() + 1e-37, "dz")
