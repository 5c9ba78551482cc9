"""The 8-bit decode's bounded wait: it gives up after its limit, says so, ends early once another has given up, and waits for nothing
that has happened.  One warp on a barrier of its own; the limit is 2^14 cycles."""
import time

import pytest
import torch

import chunked_state_scan_causal_gb300 as la

pytestmark = pytest.mark.gpu


def test_short_wait_gives_up():
    from chunked_state_scan_causal_gb300 import build
    build.build()
    out = torch.full((10,), 9, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert la.linattn_diag_wait(out.data_ptr(), torch.cuda.current_stream().cuda_stream) == la.OK
    got = out.tolist()
    assert time.perf_counter() - t0 < 0.5
    assert got == [0, 1, la.ERR_DEVICE_TIMEOUT, 0, 1, 7, 1, 1, 7, 9]
    assert la.linattn_diag_wait(None, None) == la.ERR_INVALID
    assert la.linattn_diag_wait(out.data_ptr() + 2, None) == la.ERR_ALIGN
