"""GPU tests of shared-prefix attention where it could go wrong: a wait that runs out.
Helpers and the definition are those of test_gpu_prefix and prefix_testlib."""
import pytest
import torch

from calibration_free_vector_b200 import nsn
from test_gpu_prefix import SCALE, books, decode, make, own_counts, queries, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,g,dt,cap", [(4, 4, torch.bfloat16, None), (70, 8, torch.float16, None),
                                        (64, 4, torch.float32, 2304)])     # (the last: own parts by the decode kernel)
def test_a_wait_that_runs_out_gives_nan_and_a_status_bit(B, g, dt, cap):
    # one CTA gives up; the table entries and partials that it would have written are never read
    H = 2
    caches = make([(2560, 100), (1280, 0)], own_counts(B, H), 2, 1, False, seed=101, cap=cap)
    _, _, dk, dv = books(2, 1)
    q = queries((B, H * g, 128), dt, 22)
    want = decode(caches, q, dk, dv)
    ws = workspace(caches[0], caches[2], H * g)
    status = caches[2].status
    for cta in (0, 3, 1):
        out = torch.zeros_like(q)
        nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, out, ws, cta=cta)
        torch.cuda.synchronize()
        assert int(status.item()) == 2
        assert torch.isnan(out).all()
        status.zero_()
        nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws)     # the same workspace serves the next call
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert torch.equal(out, want)
    out = torch.zeros_like(q)
    nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, out, ws, cta=10**6)     # no such CTA: an ordinary call
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_give_up_refuses_a_negative_cta():
    caches = make([(128, 3)], [[(128, 3)]], 2, 2, False, seed=89)
    _, _, dk, dv = books(2, 2)
    q = queries((1, 4, 128), torch.bfloat16, 1)
    with pytest.raises(nsn.NsnError):
        nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, torch.empty_like(q),
                                        workspace(caches[0], caches[2], 4), cta=-1)
