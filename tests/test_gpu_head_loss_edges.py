"""Edges of the tied head's losses: waits that run out, and inputs at the ends of the range the entry
points allow. Bounds are derived where they are used; u = 2^-23 is one unit of a float32 sum."""
import math
import time

import pytest
import torch

from test_gpu_head_loss import BF16, DEV, F32, gen, h, mmf, operands  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


# a dx tile sums over 500 and 256 k-blocks of words before its accumulator is handed over, tens of
# microseconds; a wait polls the cap every 16 tries of about a microsecond each
@pytest.mark.parametrize("m,d,v", [(2000, 2048, 32000), (60, 4096, 65536)])
def test_waits_that_run_out_end_in_order(mmf, m, d, v):  # noqa: F811
    x, t, g = operands(71, m, d, v, BF16, BF16)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(m, generator=g, device=DEV)
    loss, lse = mmf.lm_head_xent_fwd(x, t, targets)
    want = mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    for _ in range(5):
        mmf.set_wait_limit(1)
        start = time.monotonic()
        try:
            mmf.lm_head_xent_fwd(x, t, targets)
            mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
            status = mmf.sync_status(DEV)
        finally:
            mmf.set_wait_limit(0)
        # ended by copies that landed, not by the 1 s cap of a barrier that nothing completes
        assert time.monotonic() - start < 0.9
        assert status == mmf.MMF_ERR_TIMEOUT
        again = mmf.lm_head_xent_fwd(x, t, targets)
        got = mmf.lm_head_xent_backward(x, t, targets, again[1], dloss)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert mmf.sync_status(DEV) == mmf.MMF_OK
