"""Attention over a cache in 4 bits whose expanded keys and values are made for some sequences and key heads at a time."""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from qcache_util import D, empty_cache, rows_of
from test_gpu_mixers import NAN, cu_of, gen_of, rand
from test_gpu_qcache import BITS, check, i64, many_rows, ref_attn

pytestmark = pytest.mark.gpu


# 19 sequences with both heads at a time; one with one head
CASES = [(40, 2, 16, 200_000), (2, 3, 6, 10_000_000)]


@pytest.mark.parametrize("n,hk,hq,room", CASES)
def test_sequences_in_several_turns(n, hk, hq, room):
    g = gen_of(n)
    lens_q = [(0, 1, 7, 70)[i % 4] for i in range(n)] if n > 2 else [200, 130]
    lens_k = [lens_q[i] + (211 * i) % 1500 for i in range(n)]
    T = sum(lens_q)
    cache = empty_cache(n, room, hk)
    for i, lk in enumerate(lens_k):
        cache[i, :lk] = rows_of(rand(g, lk, hk, D), rand(g, lk, hk, D))
    assert many_rows(T, n, cache, hq)
    q, lse = rand(g, T + 2, hq, D), torch.full((T + 2, hq), NAN, device="cuda")
    out = torch.full((T + 2, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    call = lambda lens, **kw: kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens), lse=lse, cu_seqlens_q=cu_of(lens_q), **kw)
    ws = call(lens_k)
    assert kda.kda_read_device_status(ws) == 0
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), True, T)
    assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()
    first = out.clone()
    call(lens_k, workspace=ws.fill_(255))
    assert torch.equal(first[:T], out[:T])
    # lengths that contradict the tensors, in the first or the last turn's sequences: no turn writes anything
    for at in (0, n - 1):
        bad = [room + 1 if i == at else lk for i, lk in enumerate(lens_k)]
        out.fill_(NAN)
        lse.fill_(NAN)
        call(bad, workspace=ws)
        assert kda.kda_read_device_status(ws) == BITS and torch.isnan(out).all() and torch.isnan(lse).all()
    # the same queries a sequence
    each = 20 if n > 2 else 160
    q, out = rand(g, n * each, hq, D), torch.full((n * each, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    assert many_rows(n * each, n, cache, hq)
    kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k))
    check(out, None, ref_attn(q, cache, 0.1, [each] * n, lens_k), True, n * each)
