"""Appending to a cache in 4 bits where there are so many rows that a warp takes four heads of a token: the same bytes as
exact arithmetic, with heads left over behind the fours, several rows of blocks, hard numbers among easy ones, and bad lengths."""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from qcache_util import D, empty_cache, fractions_of, rows_of, values_of
from test_gpu_mixers import NAN, U, cu_of, gen_of, rand
from test_gpu_qcache import i64, placed, special_vectors

pytestmark = pytest.mark.gpu


def tokens_for(hk):
    """So many that every SM has 16 warps of four (token, head) rows each."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-64 * sms // hk)


@pytest.mark.parametrize("order", ["heads", "rows", "padded"])
@pytest.mark.parametrize("hk", [1, 2, 3, 4, 5, 8, 9])
def test_append_of_many_rows_writes_the_exact_codes(hk, order):
    g = gen_of(hk)
    T = tokens_for(hk) + 3
    lens_q = [T // 2, 0, 1, T - T // 2 - 1]
    lens_k = [lens_q[0] + 5, 4, 1, lens_q[3]]
    k = rand(g, T + 2, hk, D, mul=3.0) + rand(g, hk, D, mul=2.0)
    v = rand(g, T + 2, 3 * hk * D)[:, hk * D:2 * hk * D].unflatten(1, (hk, D))
    cache = empty_cache(4, max(lens_k) + 2, hk, order)
    want = placed(cache, rows_of(k[:T], v[:T]), lens_q, lens_k)
    whole = torch.as_strided(cache, (cache.untyped_storage().nbytes(),), (1,), 0)
    gaps = whole.clone()
    torch.as_strided(gaps, cache.shape, cache.stride()).copy_(want)
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    ko, vo = (torch.full((T + 2, hk, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    args = dict(cu_seqlens=cu_of(lens_q), status=status)
    kda.kda_qcache_append(k, v, cache, i64(lens_k), k_out=ko, v_out=vo, **args)
    assert kda.kda_read_device_status(status) == 0
    assert torch.equal(whole, gaps)                                      # the rows, and nothing between them
    for ref, xo in zip(values_of(rows_of(k[:T], v[:T])), (ko, vo)):
        assert ((xo[:T].double() - ref).abs() <= U * 1.0001 * ref.abs()).all()
        assert torch.isnan(xo[T:]).all()                                 # rows behind the last sequence
    k2, v2 = k.clone(), v.clone()                                        # in place, and without the values
    kda.kda_qcache_append(k2, v2, cache.fill_(1), i64(lens_k), k_out=k2, v_out=v2, **args)
    assert torch.equal(k2[:T], ko[:T]) and torch.equal(v2[:T], vo[:T]) and torch.equal(k2[T:], k[T:]) and torch.equal(v2[T:], v[T:])
    again = empty_cache(4, max(lens_k) + 2, hk, order)
    kda.kda_qcache_append(k, v, again, i64(lens_k), **args)
    assert torch.equal(again, want)
    single = empty_cache(1, T, hk, order)                                # one sequence, without cu_seqlens
    kda.kda_qcache_append(k[:T], v[:T], single, i64([T]))
    assert torch.equal(single[0], rows_of(k[:T], v[:T]))


@pytest.mark.parametrize("hk", [4, 5])
def test_append_of_hard_numbers_among_many_rows_is_exact(hk):
    """Rows that take the long way beside rows that do not, in every place of a group of four heads."""
    x = special_vectors()
    m, expect = x.shape[0], []
    for row in x:
        codes, scale, zero = fractions_of(row)
        c = torch.tensor(codes, dtype=torch.uint8)
        expect.append((c[0::2] | c[1::2] << 4, torch.tensor([float(scale), float(zero)]).bfloat16()))
    codes, numbers = torch.stack([e[0] for e in expect]), torch.stack([e[1] for e in expect])
    T = tokens_for(hk)
    g = torch.Generator().manual_seed(hk)
    pick = torch.randint(0, m, (4, T, hk), generator=g)                  # key's halves, value's halves
    pick[:, ::2][:, :, torch.arange(hk) % 3 > 0] = 4                     # (half of the tokens mostly with easy rows: 0, 1/4, 2/4, ...)
    k, v = (torch.cat([x[pick[2 * i]], x[pick[2 * i + 1]]], -1).cuda() for i in range(2))
    want = torch.cat([codes[p] for p in pick] + [numbers[p].contiguous().view(torch.uint8) for p in pick], -1).cuda()
    for values in (False, True):
        cache = empty_cache(1, T, hk)
        out = dict(k_out=torch.empty_like(k), v_out=torch.empty_like(v)) if values else {}
        kda.kda_qcache_append(k, v, cache, i64([T]), **out)
        assert torch.equal(cache[0], want)
        if values:
            for ref, xo in zip(values_of(want), (out["k_out"], out["v_out"])):
                near = ref.abs() < 3e38                                  # (next to bf16's largest the sum may round to infinity)
                assert ((xo.double() - ref).abs() <= U * 1.0001 * ref.abs() + 2.0 ** -133)[near].all()


def test_append_of_bad_values_among_many_rows_reads_as_nan():
    hk = 5
    T, g = tokens_for(hk), gen_of(6)
    k, v = rand(g, T, hk, D), rand(g, T, hk, D)
    want = rows_of(k, v)
    at = [(1, 0, 70, NAN), (2, 3, 0, float("inf")), (3, 4, 64, -float("inf"))]
    for t, h, c, bad in at:
        k[t, h, c] = bad
    cache = empty_cache(1, T, hk, fill=0)
    kda.kda_qcache_append(k, v, cache, i64([T]))
    gk, gv = values_of(cache[0])
    hurt = torch.zeros(T, hk, D, dtype=torch.bool, device="cuda")
    for t, h, c, _ in at:
        hurt[t, h, c // 64 * 64:c // 64 * 64 + 64] = True
    assert torch.equal(torch.isnan(gk), hurt) and torch.isfinite(gv).all()
    ref = values_of(want)
    assert torch.equal(gk[~hurt], ref[0][~hurt]) and torch.equal(gv, ref[1])


@pytest.mark.parametrize("lens_k,bad", [([5000, 5000, 9000], [0]), ([9000, 4999, 9000], [1]), ([9000, 9000, 9001], [2]), ([-1, 9000, 1 << 62], [0, 2])])
def test_append_of_many_rows_with_bad_lengths(lens_k, bad):
    hk, lens_q, room = 5, [5001, 5000, 4000], 9000
    assert sum(lens_q) >= tokens_for(hk)
    g = gen_of(12)
    k, v = rand(g, sum(lens_q), hk, D), rand(g, sum(lens_q), hk, D)
    cache = empty_cache(3, room, hk, fill=7)
    want, rows = cache.clone(), rows_of(k, v)
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        if n not in bad:
            want[n, lk - lq:lk] = rows[sum(lens_q[:n]):sum(lens_q[:n + 1])]
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    kda.kda_qcache_append(k, v, cache, i64(lens_k), cu_seqlens=cu_of(lens_q), status=status)
    assert kda.kda_read_device_status(status) == kb.KDA_DEVERR_CU_SEQLENS
    assert torch.equal(cache, want)
