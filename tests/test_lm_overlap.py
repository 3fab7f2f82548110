"""Buffers that start and end at the same bytes but whose rows lie elsewhere:
an output in place has to be its input row for row (no GPU: refused before a
launch)."""
from __future__ import annotations

import ctypes as ct

import pytest

from l2_row_b200 import ds

A = 1 << 32


def at(i: int) -> int:
    return A + (i << 28)


def lseg(**kw):
    s = ds.ds_lseg(x=at(0), ids=at(1), lse=at(2), dlogp=at(3), dx=at(4), rows=2, cols=16, ld=16, ld_d=16, scale=1.0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def same_bytes(rows, cols, size, ld, size2):
    """Another leading dimension whose matrix of `size2`-byte values ends where that of `size` bytes does."""
    ld2, rest = divmod(((rows - 1) * ld + cols) * size // size2 - cols, rows - 1)
    assert rest == 0 and ld2 >= cols and ld2 * size2 != ld * size
    return ld2


@pytest.mark.parametrize("rows,ld", [(2, 48), (3, 40), (5, 72)])
def test_logit_gradient_of_a_wider_type_over_the_logits(rows, ld):
    cols = {2: 16, 3: 16, 5: 32}[rows]
    s = lseg(dx=at(0), rows=rows, cols=cols, ld=ld, ld_d=same_bytes(rows, cols, 2, ld, 4))
    assert ds.lib().ds_logp_rows_backward((ds.ds_lseg * 1)(s), 1, ds.DS_BF16, ds.DS_F32, None) == ds.DS_ERR_OVERLAP


@pytest.mark.parametrize("side", ["q", "k"])
def test_head_gradients_of_a_wider_type_over_those_of_the_output(side):
    kw = dict(pos=at(8), inv_freq=at(9), rows=2, head_dim=16, rot_dim=16)
    if side == "q":
        s = ds.ds_qngseg(q=at(0), dq_out=at(1), dq=at(1), hq=1, ld_q=16, ld_dqo=48, ld_dq=16, **kw)
    else:
        s = ds.ds_qngseg(k=at(0), dk_out=at(1), dk=at(1), hk=1, ld_kv=16, ld_dko=48, ld_dk=16, **kw)
    st = ds.lib().ds_qk_norm_rows_backward((ds.ds_qngseg * 1)(s), 1, ds.DS_BF16, ds.DS_F32, ct.c_float(1e-6), None, None,
                                           None, 0, None)
    assert st == ds.DS_ERR_OVERLAP


@pytest.mark.parametrize("with_v", [False, True])
def test_keys_in_place_of_a_cache_of_another_pitch(with_v):
    """Three rows 64 columns apart, a cache of five rows 32 apart."""
    s = ds.ds_qnseg(k=at(0), k_cache=at(0), pos=at(8), inv_freq=at(9), rows=3, cache_rows=5, hk=1, head_dim=16, rot_dim=16,
                    ld_kv=64, ld_cache=32)
    if with_v:
        s.k_cache, s.v, s.v_cache = at(1), at(2), at(2)
    assert ds.lib().ds_qk_norm_rows((ds.ds_qnseg * 1)(s), 1, ds.DS_BF16, ct.c_float(1e-6), None) == ds.DS_ERR_OVERLAP
