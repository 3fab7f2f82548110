"""The logit gradient under a large loss scale: masked logits have gradient 0
whatever the size of the factors, the others their formula's value.

Bound per value p (A - dH (z - lse)): p within (|z - lse| + 4) 2^-24 + 2^-22 of
its value, the bracket's three products and sums 4 roundings of their sizes."""
from __future__ import annotations

import math

import pytest
import torch

from l2_row_b200 import ds
from tests.lm_util import DT, U32, gen, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("factor", [1.0, 1e9, 1e24, -1e33])
@pytest.mark.parametrize("mask", [-math.inf, -1e30, "lowest"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_masked_logits(factor, mask, t):
    R, V, g = 5, 1003, gen(4)
    low = torch.finfo(DT[t]).min if mask == "lowest" else mask
    x = torch.randn(R, 1008, generator=g, device="cuda").to(DT[t])[:, :V]
    hidden = torch.rand(R, V, generator=g, device="cuda") < 0.3
    x[hidden] = low
    z = x.double()
    lse = torch.logsumexp(z, 1).float()
    lp = z - lse.double()[:, None]
    p = lp.exp()
    H = -torch.where(p > 0, p * lp, 0.0).sum(1).float()
    ids = (~hidden).int().argmax(1)
    dlogp = torch.rand(R, generator=g, device="cuda") * factor
    dH = torch.rand(R, generator=g, device="cuda") * factor
    dx = torch.full((R, 1004), 7.0, device="cuda")[:, :V]
    ds.ds_logp_rows_backward([ds.LSeg(x=x, ids=ids, lse=lse, entropy=H, dlogp=dlogp, dentropy=dH, dx=dx)], t, "f32")
    a, h = dlogp.double()[:, None], dH.double()[:, None]
    part = torch.where(p > 0, lp + H.double()[:, None], 0.0)
    want = -p * a - h * p * part
    size = p * (a.abs() + h.abs() * (part.abs() + H.double()[:, None]))
    hot = torch.nn.functional.one_hot(ids.long(), V).double() * a
    rel = (torch.where(p > 0, lp.abs(), 0.0) + 8) * U32 + 2.0 ** -22
    within(dx, want + hot, rel * size + 2 * U32 * hot.abs() + 2.0 ** -126 * (a.abs() + 128 * h.abs()), f"{factor} {mask}")
    assert bool((dx[hidden] == 0).all())
