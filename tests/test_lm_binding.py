"""What the binding of the language-model rows takes and refuses (CPU tensors
pass every check but that of the device), and calls that need a GPU."""
from __future__ import annotations

import pytest
import torch

from l2_row_b200 import ds
from tests.lm_util import gen


def test_a_call_looks_only_at_what_it_reads():
    """One segment for both directions: bf16 rows, fp32 gradients, each with a leading dimension of its own."""
    T, V, C = 3, 5, 16
    s = ds.ESeg(w=torch.zeros(V, C), ids=torch.zeros(T, dtype=torch.int64), y=torch.zeros(T, C, dtype=torch.bfloat16),
                dy=torch.zeros(T, 24)[:, :C], grad_w=torch.zeros(V, C))
    with pytest.raises(ValueError, match="lies on cpu"):
        ds.ds_embed_rows([s], "f32", "bf16")
    with pytest.raises(ValueError, match="lies on cpu"):
        ds.ds_embed_rows_backward([s], "f32", "f32")
    with pytest.raises(ValueError, match="y: expected float32"):
        ds.ds_embed_rows([s], "f32", "f32")
    with pytest.raises(ValueError, match="dy: expected bfloat16"):
        ds.ds_embed_rows_backward([s], "f32", "bf16")
    with pytest.raises(ValueError, match="share a leading dimension"):
        s.to_c()


@pytest.mark.parametrize("seg", [ds.QNSeg, ds.QNGSeg])
@pytest.mark.parametrize("D", [0, -16])
def test_head_sizes_below_one(seg, D):
    with pytest.raises(ValueError, match="head_dim"):
        seg(D, q=torch.zeros(2, 32)).to_c()


@pytest.mark.gpu
def test_one_segment_for_both_directions():
    T, V, C, g = 40, 50, 96, gen(1)
    w = torch.randn(V, C, generator=g, device="cuda")
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    dy = torch.randn(T, 104, generator=g, device="cuda")[:, :C]
    s = ds.ESeg(w=w, ids=ids, y=torch.empty(T, C, dtype=torch.bfloat16, device="cuda"), dy=dy, grad_w=torch.empty_like(w))
    ds.ds_embed_rows([s], "f32", "bf16")
    ds.ds_embed_rows_backward([s], "f32", "f32")
    assert torch.equal(s.y, w[ids].bfloat16())
    want = torch.zeros(V, C, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    assert bool(((s.grad_w - want).abs() <= 40 * 2.0 ** -24 * 5).all())      # at most 40 terms below 5
