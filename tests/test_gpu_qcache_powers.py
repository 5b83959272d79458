"""Attention of many rows over a cache in 4 bits whose values differ by powers of two from key to key: what a large value does
to the others goes by its weight alone.

The bounds are those of test_gpu_qcache.py and one more term.  A weight times its value's power of two is rounded to fp16 as well where
it falls below fp16's normal numbers, by at most 2^-25 there.  The largest such product of a row is at least 2^-10 of what
stands for 2^7: a reference that is rounded up (2^1), powers that a block of keys may share (2^9).  With R the largest product of a weight
and its key's largest value, key j moves channel c by at most 2^-25 2^-7 2^10 R |v_jc| / max_c |v_jc|, twice
that since a power of two is up to half of the number it stands for: 2^-21 R sum_j |v_jc| / max_c |v_jc|.
"""
import math

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from qcache_util import D, empty_cache, rows_of, values_of
from test_gpu_mixers import NAN, U, cu_of, gen_of, rand
from test_gpu_qcache import i64, many_rows, ref_attn

pytestmark = pytest.mark.gpu


def weights_below_normal(q, cache, scale, lens_q, lens_k):
    """2^-21 R sum_j |v_jc| / max_c |v_jc| for every query, head and channel."""
    hq, hk = q.shape[1], cache.shape[2]
    out = torch.zeros(sum(lens_q), hq, D, dtype=torch.float64, device="cuda")
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        for h in range(hk):
            k, v = values_of(cache[n, :lk, h])
            g = slice(h * hq // hk, (h + 1) * hq // hk)
            w = torch.einsum("ihd,jd->hij", q[a:a + lq, g].double(), k) * scale
            seen = torch.arange(lk, device="cuda") <= torch.arange(lq, device="cuda")[:, None] + lk - lq
            p = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
            top = v.abs().amax(-1)
            most = (p * top).amax(-1)
            share = v.abs() / torch.where(top > 0, top, 1.0)[:, None]
            out[a:a + lq, g] = torch.einsum("hi,ij,jc->ihc", most, seen.double(), share)
        a += lq
    return 2.0 ** -21 * out


LOW = -4.0     # keys of this number score some 50 below the others (queries lie around 1)


def keys_and_values(g, kind, r, lk, hk):
    k, v = rand(g, lk, hk, D, mul=0.25).float(), rand(g, lk, hk, D).float()
    at = torch.arange(lk, device="cuda")
    if kind == "blocks":            # large values without weight, a block of keys in five
        large = at // 128 % 5 == 0
        k[large] = LOW
        v[~large] *= 2.0 ** -r
    elif kind == "rows":            # one large value without weight among ordinary ones, five blocks apart
        large = at % 640 == 77
        k[large] = LOW
        v[large] *= 2.0 ** r
    elif kind == "later":           # a large value that the last two queries see only
        v[lk - 2] *= 2.0 ** r
    elif kind == "sink":            # a key of nearly all weight and next to no value, five blocks apart
        k[at % 640 == 3] = 1.0
        v[at % 640 == 3] *= 2.0 ** -r
    elif kind == "mixed":           # every key its own power
        v *= torch.exp2(torch.randint(-r // 2, r // 2 + 1, (lk, 1, 1), generator=g, device="cuda").float())
    elif kind == "steps":           # ... every block its own
        v *= torch.exp2(((at // 128 * 5 % 7 - 3) * r // 6).float())[:, None, None]
    elif kind == "zeros":           # values of zero among the others, whole blocks of them too
        v[(at % 3 == 0) | (at // 128 % 4 == 1)] = 0.0
        v[at % 640 == 10] *= 2.0 ** r
        k[at % 640 == 10] = LOW
    return k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("r", [4, 9, 12, 16, 20, 24, 30, 40])
@pytest.mark.parametrize("kind", ["blocks", "rows", "later", "sink", "mixed", "steps", "zeros"])
@pytest.mark.parametrize("lens_q,lens_k", [([300], [5000]), ([40, 260, 90], [333, 2500, 90])])
def test_values_of_different_powers(lens_q, lens_k, kind, r):
    g = gen_of(100 + r)
    hq, hk, T, scale = 32, 2, sum(lens_q), 0.1
    cache = empty_cache(len(lens_k), 5001, hk)
    assert many_rows(T, len(lens_q), cache, hq)
    for n, lk in enumerate(lens_k):
        cache[n, :lk] = rows_of(*keys_and_values(g, kind, r, lk, hk))
    q = (rand(g, T, hq, D).float() + 1.0).bfloat16()
    out, lse = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, scale, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    assert kda.kda_read_device_status(ws) == 0
    ref, size, spread, moved, rlse, most = ref_attn(q, cache, scale, lens_q, lens_k)
    bound = 1.01 * (U * ref.abs() + 2.0 ** -10 * size + U * U * moved) + 2.0 ** -14 * (size + spread + moved) + 1e-30
    bound += weights_below_normal(q, cache, scale, lens_q, lens_k)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), f"{(err / bound).max().item():.3g} of its bound, {(err > bound).sum().item()} of {err.numel()}"
    assert ((lse.double() - rlse).abs() <= 2.0 ** -14 * (1 + most)).all()


@pytest.mark.parametrize("r", [16, 24, 40])
def test_an_early_token_does_not_depend_on_later_values(r):
    """The last keys' values, enlarged, change the queries that see them only: the others to the rounding of their results
    (their weights, between powers of two that may lie elsewhere, are rounded by no more than before)."""
    g = gen_of(7)
    hq, hk, lq, lk = 32, 2, 300, 3000
    k, v = keys_and_values(g, "none", 0, lk, hk)
    q = (rand(g, lq, hq, D).float() + 1.0).bfloat16()
    outs = []
    for power in (0, r):
        v2 = v.clone()
        v2[lk - 20:] *= 2.0 ** power
        cache = empty_cache(1, 5001, hk)
        cache[0, :lk] = rows_of(k, v2)
        assert many_rows(lq, 1, cache, hq)
        out = torch.empty(lq, hq, D, dtype=torch.bfloat16, device="cuda")
        kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64([lk]))
        outs.append(out[:lq - 20].double())
    cache = empty_cache(1, lk, hk)
    cache[0] = rows_of(k, v)
    ref, size, _, moved, _, _ = (x[:lq - 20] for x in ref_attn(q, cache, 0.1, [lq], [lk]))
    below = weights_below_normal(q, cache, 0.1, [lq], [lk])[:lq - 20]
    bound = 1.01 * (U * ref.abs() + 2.0 ** -10 * size + U * U * moved) + 2.0 ** -14 * (size + moved) + below
    for out in outs:
        assert ((out - ref).abs() <= bound).all()


@pytest.mark.parametrize("r", [9, 16, 24, 40])
@pytest.mark.parametrize("kind", ["blocks", "rows", "later", "sink", "mixed", "steps", "zeros"])
@pytest.mark.parametrize("lens_q,lens_k", [([1, 1], [5000, 333]), ([4, 1, 2], [2500, 90, 700])])
def test_few_rows_over_values_of_different_powers(lens_q, lens_k, kind, r):
    """The same without expansion, where weights carry their values' scales in bf16 and so have powers enough."""
    g = gen_of(200 + r)
    hq, hk, T, scale = 32, 8, sum(lens_q), 0.1
    cache = empty_cache(len(lens_k), 5001, hk)
    assert not many_rows(T, len(lens_q), cache, hq)
    for n, lk in enumerate(lens_k):
        cache[n, :lk] = rows_of(*keys_and_values(g, kind, r, lk, hk))
    q = (rand(g, T, hq, D).float() + 1.0).bfloat16()
    out, lse = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, scale, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    assert kda.kda_read_device_status(ws) == 0
    ref, size, spread, moved, rlse, most = ref_attn(q, cache, scale, lens_q, lens_k)
    bound = 1.01 * (U * ref.abs() + U * spread) + 2.0 ** -14 * (size + spread + moved) + 1e-30
    err = (out.double() - ref).abs()
    assert (err <= bound).all(), f"{(err / bound).max().item():.3g} of its bound, {(err > bound).sum().item()} of {err.numel()}"
    assert ((lse.double() - rlse).abs() <= 2.0 ** -14 * (1 + most)).all()
