"""Run only by the child process of tests/test_gpu_qcache_timeout.py, against the test-only build
libkda_waittest.so (the file name keeps it out of the normal collection).

That build gives up a bounded wait after a few milliseconds and, when KDA_TEST_SKIP_SHARE names a share, has that
share of the attention over a 4-bit cache wait in vain: few rows, for a copy that was never started; many rows, for weights
that are never announced, in the first of the call's launches.  The call must come back with KDA_DEVERR_TIMEOUT set and the
context must stay usable: the next call, without the skip, is right.
"""
import os

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from qcache_util import D, empty_cache, rows_of
from test_gpu_mixers import NAN, cu_of, gen_of, rand
from test_gpu_qcache import check, filled, i64, many_rows, ref_attn

pytestmark = pytest.mark.gpu


def with_share(share, call):
    assert os.path.basename(kb.library_path()) == "libkda_waittest.so"
    os.environ["KDA_TEST_SKIP_SHARE"] = str(share)
    try:
        return kda.kda_read_device_status(call())
    finally:
        del os.environ["KDA_TEST_SKIP_SHARE"]


def run(cache, lens_q, lens_k, hq, share, want):
    g, T = gen_of(52), sum(lens_q)
    q, out = rand(g, T, hq, D), torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, hq), NAN, device="cuda")
    many = many_rows(T, len(lens_q), cache, hq)
    ws = torch.full((kda.kda_attn_qcache_workspace_size(T, hq, cache.shape[2], len(lens_q), cache.shape[1]),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q), workspace=ws)
    ref = ref_attn(q, cache, 0.1, lens_q, lens_k)
    for _ in range(3):
        assert with_share(share, call) & want
        assert kda.kda_read_device_status(call()) == 0
        check(out, lse, ref, many, T)
    return many


# tiles of 8 and of 16 rows, one key head and two together; pieces of many slices, and many pieces of few
@pytest.mark.parametrize("share", [2, 40, 74, 100])
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,order", [
    ([1, 1], [9000, 3000], 8, 2, "heads"), ([4] * 3, [3000, 9000, 700], 32, 8, "heads"), ([1] * 32, [500 + 37 * i for i in range(32)], 32, 8, "rows"),
    ([4] * 20, [300 + 61 * i for i in range(20)], 32, 8, "heads"), ([1] * 200, [40 + i for i in range(200)], 32, 8, "heads")])
def test_few_rows_whose_copy_never_comes(lens_q, lens_k, hq, hk, order, share):
    assert not run(filled(gen_of(51), lens_k, hk, order), lens_q, lens_k, hq, share, kb.KDA_DEVERR_TIMEOUT)


@pytest.mark.parametrize("share", [3, 100])
@pytest.mark.parametrize("lens_q,lens_k", [([700, 60], [3700, 60]), ([130] * 4, [2000, 130, 700, 3000])])
def test_many_rows_whose_weights_never_come(lens_q, lens_k, share):
    assert run(filled(gen_of(51), lens_k, 8, "heads", room=4000), lens_q, lens_k, 32, share, kb.KDA_DEVERR_TIMEOUT)


@pytest.mark.parametrize("share,want", [(3, kb.KDA_DEVERR_TIMEOUT), (-2, kb.KDA_DEVERR_INTERNAL), (-2 - 151, kb.KDA_DEVERR_INTERNAL)])
def test_a_report_of_the_first_of_several_turns_is_not_lost(share, want):
    """Three of eight key heads at a time: what the first launch reports is still there after the last."""
    lens_q, lens_k, hk, g = [300, 200], [20000, 9000], 8, gen_of(53)
    cache = empty_cache(2, 260_000, hk)
    for i, lk in enumerate(lens_k):
        cache[i, :lk] = rows_of(rand(g, lk, hk, D), rand(g, lk, hk, D))
    assert run(cache, lens_q, lens_k, 16, share, want)
