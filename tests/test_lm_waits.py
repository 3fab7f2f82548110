"""Waits that run out: with a limit of zero any wait of a kernel for a copy
that is on its way may give up.  The call then reports it, nothing hangs or is
left behind, and the next call with the usual limit gives the usual bits."""
from __future__ import annotations

import pytest
import torch

from l2_row_b200 import ds
from tests.lm_util import gen

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000_000


@pytest.fixture
def no_patience():
    def set_limit(on):
        ds.ds_debug_set_wait_limit_ns(0 if on else LIMIT_NS)

    yield set_limit
    ds.ds_debug_set_wait_limit_ns(LIMIT_NS)


def check(run, no_patience):
    want = run()
    assert ds.ds_get_device_status() == ds.DS_OK
    for _ in range(5):
        no_patience(True)
        got = run()
        status = ds.ds_get_device_status()
        no_patience(False)
        assert status in (ds.DS_OK, ds.DS_ERR_DEVICE_TIMEOUT)
        if status == ds.DS_OK:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        again = run()
        assert ds.ds_get_device_status() == ds.DS_OK
        assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("R,V", [(1, 131072), (20, 60001), (700, 20000), (900, 4000)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_log_probabilities(R, V, t, no_patience):
    """A cluster a row, clusters of fewer CTAs, many rows a CTA, short rows."""
    g = gen(7)
    x = torch.randn(R, -(-V // 8) * 8, generator=g, device="cuda").to(torch.float32 if t == "f32" else torch.bfloat16)[:, :V]
    ids = torch.randint(0, V, (R,), generator=g, device="cuda")

    def run():
        o = [torch.zeros(R, device="cuda") for _ in range(3)]
        top = torch.zeros(R, 20, dtype=torch.int32, device="cuda")
        ds.ds_logp_rows([ds.LSeg(x=x, ids=ids, logp=o[0], lse=o[1], entropy=o[2], top_id=top)], t)
        return [*o, top]

    check(run, no_patience)


@pytest.mark.parametrize("C", [768, 4096])
def test_embedding_gradient(C, no_patience):
    g = gen(8)
    V, T = 3000, 5000
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[: T // 4] = 5
    w, dy = torch.randn(V, C, generator=g, device="cuda"), torch.randn(T, C, generator=g, device="cuda")

    def run():
        gw = torch.zeros(V, C, device="cuda")
        ds.ds_embed_rows_backward([ds.ESeg(w=w, ids=ids, dy=dy, grad_w=gw, unit=True)], "f32", "f32")
        return [gw]

    check(run, no_patience)
