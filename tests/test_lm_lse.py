"""The log-sum-exp against 64 bits where it is large: one rounding of the
result, not one for every factor of it.

Bound: half a step of the result, and what the sum of exponentials carries
whatever the result's size: (40 + steps) 2^-24 for its depth and 2^-22 for the
exp2 unit as in test_lm_logp.py, its terms' exponents (of a product with a factor
within 2^-23 of scale log2 e, and a rounding of their own) at most 60 away
from the maximum wherever they count: 4 x 60 x 2^-24."""
from __future__ import annotations

import pytest
import torch

from l2_row_b200 import ds
from tests.lm_util import U32, gen, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V", [(300, 2001), (300, 9001), (9, 40001)])
@pytest.mark.parametrize("scale", [0.37, 0.8, 1.0, 1.3])
@pytest.mark.parametrize("shift", [-1e5, -1000.0, 40.0, 1000.0, 1e5])
def test_large_values(R, V, scale, shift):
    ld = -(-V // 4) * 4
    x = (torch.randn(R, ld, generator=gen(3), device="cuda") * 3 + shift)[:, :V]
    lse = torch.empty(R, device="cuda")
    ds.ds_logp_rows([ds.LSeg(x=x, lse=lse, scale=scale)], "f32")
    want = torch.logsumexp(x.double() * float(torch.tensor(scale, dtype=torch.float32)), 1)
    within(lse, want, (40 + V // 2048 + 1) * U32 + 2.0 ** -22 + 4 * U32 * 60, "lse")
