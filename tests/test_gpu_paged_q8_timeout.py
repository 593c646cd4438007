"""Bounded waits of the 8-bit paged decode that run out, on a B200: the loader is kept (test hook) from
asking for the rotary columns, with a short wait limit.  The latents' copies and the products
over them are under way when the waits give up, and have to end before the kernel does: those
waits keep the default limit.  Nothing faults or hangs; each call returns and latches a timeout."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged_q8 import Decode, mla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Q,lens", [(16, 1, [700, 5]), (128, 1, [3000, 100, 64]), (128, 9, [300]), (16, 2, [40] * 400)])
def test_waits_that_run_out_latch_a_timeout_and_the_next_call_works(H, Q, lens):
    D = Decode(H, Q, lens, seed=95)
    want = D.run()
    assert mla.mla_get_device_error() == (0, 0)
    mla.mla_set_wait_limit(256)
    mla.mla_test_starve_projection(True)
    try:
        D.run()
        st, _ = mla.mla_get_device_error()
    finally:
        mla.mla_test_starve_projection(False)
        mla.mla_set_wait_limit(0)
    assert st == mla.MLA_ERR_DEVICE_TIMEOUT
    assert mla.mla_get_device_error() == (0, 0)
    assert torch.equal(D.check(f"H={H} q_len={Q} after a timeout"), want)
