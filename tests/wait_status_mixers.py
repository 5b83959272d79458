"""Run only by the child process of tests/test_gpu_mixers_wait_limit.py, against the test-only build
libkda_waittest.so (the file name keeps it out of the normal collection).

That build has one share find itself unsound (KDA_TEST_SKIP_SHARE = -2 - share): it computes nothing and reports
KDA_DEVERR_INTERNAL.  Whichever share it is, the bit has to be in the status word, and gone after the next call
on the same workspace.
"""
import os

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from test_gpu_mixers import D, cu_of, gen_of, rand

pytestmark = pytest.mark.gpu
SHARES = [0, 1, 2, 75, 150, 151]


def status_of(share, call, ws):
    assert os.path.basename(kb.library_path()) == "libkda_waittest.so"
    os.environ["KDA_TEST_SKIP_SHARE"] = str(-2 - share)
    try:
        call(ws)
    finally:
        del os.environ["KDA_TEST_SKIP_SHARE"]
    return kda.kda_read_device_status(ws)


@pytest.mark.parametrize("share", SHARES)
def test_attn_reports_an_unsound_share(share):
    g = gen_of(61)
    q, k, v = rand(g, 2000, 8, D), rand(g, 2000, 2, D), rand(g, 2000, 2, D)
    out, cu = torch.empty_like(q), cu_of([1900, 100])
    call = lambda ws: kda.kda_attn_fwd(q, k, v, 0.1, out, cu_seqlens_q=cu, workspace=ws)
    ws = torch.full((kda.kda_attn_workspace_size(2000, 8, 2),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        assert status_of(share, call, ws) == kb.KDA_DEVERR_INTERNAL
    call(ws)
    assert kda.kda_read_device_status(ws) == 0


@pytest.mark.parametrize("share", SHARES)
def test_lin_reports_an_unsound_share(share):
    g = gen_of(62)
    h, lens = 64, [400, 300]
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld, out, cu = torch.full((h,), -0.1, device="cuda"), torch.empty_like(q), cu_of(lens)
    call = lambda ws: kda.kda_lin_fwd(q, k, v, ld, 0.1, out, cu_seqlens=cu, workspace=ws)
    ws = torch.full((kda.kda_lin_workspace_size(sum(lens), h, len(lens)),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        assert status_of(share, call, ws) & ~kb.KDA_DEVERR_TIMEOUT == kb.KDA_DEVERR_INTERNAL   # (others wait for its state)
    call(ws)
    assert kda.kda_read_device_status(ws) == 0
