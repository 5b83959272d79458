"""Attention over a cache in 4 bits where keys and values are expanded first (many rows, and room for many keys): lengths
that contradict the tensors, and prompts that see what later steps see."""
import math

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from qcache_util import D, empty_cache
from test_gpu_mixers import NAN, U, cu_of, gen_of, rand
from test_gpu_qcache import BITS, check, filled, i64, many_rows, ref_attn, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens_q,lens_k", [
    ([0, 100, 200], [300, 2701]), ([0, 100, 200], [-1, 300]), ([0, 100, 201], [300, 300]), ([1, 100, 200], [300, 300]), ([0, 300, 200], [300, 300]),
    ([0, 100, 200], [1 << 40, 300]), ([0, 100, 200], [300, -(1 << 62)]), ([0, -100, 200], [300, 300]), ([0, 1 << 40, 200], [300, 300]),
    ([0, 100, 1 << 33], [300, 300]), (None, [300, 2701]), (None, [-5, 300]), (None, [1 << 31, 300])])
def test_bad_lengths(lens_q, lens_k):
    """Nothing is written, the status says so, and the next call on the workspace is right."""
    g = gen_of(12)
    hq, hk, T = 4, 2, 200
    cache = filled(g, [300, 300], hk, "heads", room=2700)
    assert many_rows(T, 2, cache, hq)
    q = rand(g, T, hq, D)
    out, lse = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=None if lens_q is None else i64(lens_q))
    assert kda.kda_read_device_status(ws) == BITS
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64([300, 300]), lse=lse, workspace=ws)
    assert kda.kda_read_device_status(ws) == 0
    check(out, lse, ref_attn(q, cache, 0.1, [100, 100], [300, 300]), True, T)


def test_prompts_see_what_later_steps_see():
    """Attention over the appended values themselves, and later over the cache, answers the same query the same way."""
    g = gen_of(42)
    lens, hq, hk = [350, 133, 1], 8, 2
    T = sum(lens)
    q, k, v = rand(g, T, hq, D), rand(g, T, hk, D), rand(g, T, hk, D)
    cache = empty_cache(3, max(wide(lens, hq), 350), hk, "rows")
    assert many_rows(T, 3, cache, hq)
    kda.kda_qcache_append(k, v, cache, i64(lens), cu_seqlens=cu_of(lens), k_out=k, v_out=v)
    a, b = (torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    kda.kda_attn_fwd(q, k, v, D ** -0.5, a, cu_seqlens_q=cu_of(lens))
    kda.kda_attn_qcache_fwd(q, cache, D ** -0.5, b, i64(lens), cu_seqlens_q=cu_of(lens))
    out, size, _, moved, _, _ = ref_attn(q, cache, D ** -0.5, lens, lens)
    # the appended values are rounded once more (keys and values, as far as the last term), the weights and results of each too
    assert ((a.double() - b.double()).abs() <= U * 1.01 * (2 * out.abs() + 2 * size + moved) + 2.0 ** -10 * size + 2.0 ** -14 * (size + moved)).all()


def test_rows_that_see_no_key_among_many():
    """More queries than keys: the first ones see nothing, whatever lies in the cache."""
    g = gen_of(43)
    lens_q, lens_k, hq, hk = [400, 150, 200], [250, 0, 129], 8, 2
    T = sum(lens_q)
    cache = filled(g, lens_k, hk, "padded", room=wide(lens_q, hq))
    assert many_rows(T, 3, cache, hq)
    q, out, lse = rand(g, T, hq, D), torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), True, T)
    assert (out[:150] == 0).all() and (lse[:150] == -math.inf).all() and (out[400:621] == 0).all()
