"""Layouts that the cache in 4 bits and its attention take and that lie apart from the usual ones: sequences inside the rows,
queries and results with the heads outside, very many sequences, a single row, keys up to the room's end."""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from qcache_util import D, ROW, empty_cache, rows_of
from test_gpu_mixers import NAN, cu_of, gen_of, rand
from test_gpu_qcache import check, i64, many_rows, ref_attn

pytestmark = pytest.mark.gpu


def fill(g, cache, lens_k):
    hk = cache.shape[2]
    k, v = rand(g, sum(lens_k), hk, D), rand(g, sum(lens_k), hk, D)
    kda.kda_qcache_append(k, v, cache, i64(lens_k), cu_seqlens=cu_of(lens_k))
    a = 0
    for n, lk in enumerate(lens_k):
        assert torch.equal(cache[n, :lk], rows_of(k[a:a + lk], v[a:a + lk]))
        a += lk


# [positions, sequences, heads], [heads, positions, sequences], [positions, heads, sequences]
@pytest.mark.parametrize("order", [(1, 0, 2, 3), (2, 1, 0, 3), (1, 2, 0, 3)])
@pytest.mark.parametrize("lens_q,lens_k,room", [([1, 1, 1], [700, 64, 33], 700), ([2, 0, 5], [90, 3, 400], 401), ([130, 90, 1], [900, 200, 77], 2400)])
def test_caches_with_the_sequences_inside(lens_q, lens_k, room, order):
    g, hq, hk, T = gen_of(61), 16, 4, sum(lens_q)
    shape = (3, room, hk, ROW)
    whole = torch.full([shape[i] for i in order], 255, dtype=torch.uint8, device="cuda")
    cache = whole.permute([order.index(i) for i in range(4)])
    assert cache.shape == shape
    fill(g, cache, lens_k)
    assert (whole == 255).all(-1).sum() == (3 * room - sum(lens_k)) * hk      # the other rows are as they were
    q, out, lse = rand(g, T, hq, D), torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    assert many_rows(T, 3, cache, hq) == (T > 100)
    kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), T > 100, T)


@pytest.mark.parametrize("lens_q,lens_k,room", [([1, 1], [700, 64], 700), ([3, 5], [90, 400], 401), ([130, 91], [900, 200], 2400)])
def test_queries_and_results_with_the_heads_outside(lens_q, lens_k, room):
    g, hq, hk, T = gen_of(62), 12, 4, sum(lens_q)
    cache = empty_cache(2, room, hk)
    fill(g, cache, lens_k)
    q = rand(g, hq, T + 1, 2 * D)[:, 1:, D:].transpose(0, 1)
    wide = torch.full((hq + 1, T + 2, 3 * D), NAN, dtype=torch.bfloat16, device="cuda")
    out = wide[1:, 1:T + 1, D:2 * D].transpose(0, 1)
    assert many_rows(T, 2, cache, hq) == (T > 100)
    kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), cu_seqlens_q=cu_of(lens_q))
    check(out, None, ref_attn(q, cache, 0.1, lens_q, lens_k), T > 100, T)
    wide[1:, 1:T + 1, D:2 * D] = NAN
    assert torch.isnan(wide).all()                                            # nothing beside the results


@pytest.mark.parametrize("tokens,n,room,hq,hk", [(1, 5000, 40, 4, 2), (3, 1500, 70, 8, 1), (60, 700, 90, 8, 2)])
def test_very_many_sequences(tokens, n, room, hq, hk):
    """More sequences than a block has threads; some without queries, some without keys."""
    g = gen_of(63)
    lens_q = [0 if i % 7 == 3 else tokens for i in range(n)]
    lens_k = [0 if i % 11 == 5 else (13 * i) % room + 1 for i in range(n)]
    cache = empty_cache(n, room, hk)
    k, v = rand(g, sum(lens_k), hk, D), rand(g, sum(lens_k), hk, D)
    kda.kda_qcache_append(k, v, cache, i64(lens_k), cu_seqlens=cu_of(lens_k))
    T = sum(lens_q)
    q, out, lse = rand(g, T, hq, D), torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    assert many_rows(T, n, cache, hq) == (tokens == 60)
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    assert kda.kda_read_device_status(ws) == 0
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), tokens == 60, T)


def test_a_cache_of_one_row():
    g = gen_of(64)
    for n, hk in ((1, 1), (5, 3)):
        cache = empty_cache(n, 1, hk)
        fill(g, cache, [1] * n)
        q, out = rand(g, n, 2 * hk, D), torch.full((n, 2 * hk, D), NAN, dtype=torch.bfloat16, device="cuda")
        kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64([1] * n))
        check(out, None, ref_attn(q, cache, 0.1, [1] * n, [1] * n), False, n)
