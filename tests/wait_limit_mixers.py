"""Run only by the child process of tests/test_gpu_mixers_wait_limit.py, against the test-only build
libkda_waittest.so (the file name keeps it out of the normal collection).

That build's waits give up 256 times sooner than the library's, whose limit is about a second: after
about 4 ms, those for memory after 4 to 10.  A call whose states never come lasts one wait for memory, then one of the
roles that wait for the one that gave up, and 2 ms of winding down.
"""
import os

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from test_gpu_mixers import D, cu_of, gen_of, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,h,share", [([1407, 94], 64, 60), ([7680], 4, 7)], ids=["two_shares", "many_shares"])
def test_waits_for_memory_have_the_limit_of_the_others(lens, h, share):
    assert os.path.basename(kb.library_path()) == "libkda_waittest.so"
    g = gen_of(52)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld, out, final = torch.full((h,), -0.1, device="cuda"), torch.empty_like(q), torch.empty(len(lens), h, D, D, device="cuda")
    cu = cu_of(lens)
    call = lambda: kda.kda_lin_fwd(q, k, v, ld, 0.1, out, final_state=final, cu_seqlens=cu)
    assert kda.kda_read_device_status(call()) == 0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    os.environ["KDA_TEST_SKIP_SHARE"] = str(share)
    try:
        start.record()
        ws = call()
        end.record()
    finally:
        del os.environ["KDA_TEST_SKIP_SHARE"]
    assert kda.kda_read_device_status(ws) & kb.KDA_DEVERR_TIMEOUT
    torch.cuda.synchronize()
    ms = start.elapsed_time(end)
    print(f"{ms:.1f} ms")
    assert ms < 25.0
