"""Run only by the child process of tests/test_gpu_mixers_timeout.py, against the test-only
build libkda_waittest.so (the file name keeps it out of the normal collection).

That build gives up a bounded wait after a few milliseconds and, when KDA_TEST_SKIP_SHARE names
a share, has that share withhold an arrival: in attention the weights of its tiles, in linear
attention the state that it publishes for the shares behind it.  The call must come back with
KDA_DEVERR_TIMEOUT set and the context must stay usable: the next call, without the skip, is right.
"""
import os

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from test_gpu_mixers import D, NAN, check_attn, check_lin_out, check_state, cu_of, gen_of, rand, ref_attn
from test_gpu_mixers_shapes import chunked_lin

pytestmark = pytest.mark.gpu


def withheld(share, call):
    assert os.path.basename(kb.library_path()) == "libkda_waittest.so"
    os.environ["KDA_TEST_SKIP_SHARE"] = str(share)
    try:
        return kda.kda_read_device_status(call())
    finally:
        del os.environ["KDA_TEST_SKIP_SHARE"]


@pytest.mark.parametrize("lens_q,lens_k", [([700, 60], [700, 60]), ([1, 1], [9000, 300])], ids=["prompts", "tokens"])
def test_attn_weights_that_never_come(lens_q, lens_k):
    g = gen_of(51)
    q, k, v = rand(g, sum(lens_q), 8, D), rand(g, sum(lens_k), 2, D), rand(g, sum(lens_k), 2, D)
    out = torch.full_like(q, NAN)
    call = lambda: kda.kda_attn_fwd(q, k, v, 0.1, out, cu_seqlens_q=cu_of(lens_q), cu_seqlens_k=cu_of(lens_k))
    assert withheld(3, call) & kb.KDA_DEVERR_TIMEOUT
    assert kda.kda_read_device_status(call()) == 0
    at = [0, lens_k[0], sum(lens_k)]
    check_attn(q, out, None, ref_attn(q, k, v, 0.1, lens_q, lens_k, lambda n: (k[at[n]:at[n + 1]], v[at[n]:at[n + 1]])), 0.1)


@pytest.mark.parametrize("lens,h,share", [([1407, 94], 64, 60), ([7680], 4, 7)], ids=["two_shares", "many_shares"])
def test_lin_states_that_never_come(lens, h, share):
    g = gen_of(52)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld = -(2.0 ** (-10.0 * torch.arange(1, h + 1) / h)).cuda()
    init, final = rand(g, len(lens), h, D, D, dtype=torch.float32), torch.full((len(lens), h, D, D), NAN, device="cuda")
    out = torch.full_like(q, NAN)
    call = lambda: kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
    assert withheld(share, call) & kb.KDA_DEVERR_TIMEOUT
    assert kda.kda_read_device_status(call()) == 0
    o, A, s, t = chunked_lin(q[0], k[0], v[0], ld, 0.1, lens, init)
    check_lin_out(out[0], o, A)
    check_state("final_state", final, s, t)
