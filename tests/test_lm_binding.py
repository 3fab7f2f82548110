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


def test_a_single_row_needs_no_leading_dimension():
    """One token's row of an odd width, as a model returns it; several such rows have to be padded."""
    x = torch.zeros(1, 50257, dtype=torch.bfloat16)
    for t in (x, x.expand(3, -1)[:1], torch.zeros(50257, 2, dtype=torch.bfloat16)[:, 0].contiguous()[None]):
        s = ds.LSeg(x=t, dx=torch.zeros(1, 50257)).to_c()
        assert (s.ld, s.ld_d, s.rows, s.cols) == (50264, 50260, 1, 50257)
    s = ds.ESeg(w=torch.zeros(1, 5), ids=torch.zeros(1, dtype=torch.int32), y=torch.zeros(1, 5, dtype=torch.bfloat16)).to_c()
    assert (s.ld, s.ld_y) == (8, 8)
    with pytest.raises(ValueError, match="columns must be contiguous"):
        ds.LSeg(x=torch.zeros(1, 6)[:, ::2]).to_c()
    assert ds.LSeg(x=torch.zeros(2, 50257)).to_c().ld == 50257


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 1003, 50257])
def test_a_single_row_of_odd_width(t, V):
    """The bits of the same row in a padded matrix; nothing is written past its end."""
    g = gen(2)
    dt = torch.float32 if t == "f32" else torch.bfloat16
    wide = torch.randn(3, V + 8 - V % 8, generator=g, device="cuda").to(dt)
    ids = torch.tensor([V - 1], device="cuda")
    outs = []
    for x, dx in ((wide[1:2, :V], torch.empty_like(wide)[:1, :V]),
                  (wide[1:2, :V].contiguous(), torch.full((V + 3,), 7.0, dtype=dt, device="cuda")[:V][None])):
        o = [torch.empty(1, device="cuda") for _ in range(3)]
        top = torch.empty(1, 1, dtype=torch.int32, device="cuda")
        ds.ds_logp_rows([ds.LSeg(x=x, ids=ids, logp=o[0], lse=o[1], entropy=o[2], top_id=top)], t)
        ds.ds_logp_rows_backward([ds.LSeg(x=x, ids=ids, lse=o[1], entropy=o[2], dlogp=o[0], dentropy=o[2], dx=dx)], t)
        outs.append((*o, top, dx.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    tail = torch.as_strided(dx, (V + 3,), (1,))[V:]
    assert bool((tail == 7).all())
    y = torch.empty(1, V, device="cuda")
    w = wide[:1, :V].contiguous()
    ds.ds_embed_rows([ds.ESeg(w=w, ids=torch.zeros(1, dtype=torch.int32, device="cuda"), y=y)], t, "f32")
    assert torch.equal(y, w.float())


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
