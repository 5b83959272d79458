"""The cache in 4 bits on the GPU: appending against exact arithmetic (equal bytes), and the attention over it
against a plain evaluation of its formulas in 64 bits.

Bounds of the attention, per element, with u = 2^-8 the unit roundoff of bf16:
  few rows     u |o| + u sum_j p_j |v_j - w_j|: the output's rounding and the weights', which take the values' scales
               with them.  w_j = zero_j + 7.5 scale_j is the middle of the value's group: the products are
               sum_j (p_j scale_j (1 + d_j)) (code_j - 7.5), |d_j| <= u, beside sum_j p_j w_j in fp32, and
               scale_j (code_j - 7.5) = v_j - w_j; so a weight's rounding moves the output by p_j d_j (v_j - w_j),
               which may be more than p_j u |v_j| where a value lies near zero and its group's middle does not.
               What the codes stand for is not rounded
  many rows    (more than 112 (token, head) rows that share a key head, on average) values and weights are rounded to fp16,
               2^-11 each: 2^-10 sum_j p_j |v_j|.  Keys and queries are exact but for what is 2^-25 of
               the largest of their block and row: a score is off by less than u^2 b_ij, b_ij = scale sum_c |q_ic k_jc|, which moves the weight p_j by p_j u^2 (b_ij + sum_k p_k b_ik)
               to first order
  both         2^-14 of those sums for fp32 (scores of up to b_ij from terms of that size, sums over the keys)
  lse          2^-14 of 1 + b_max
The Frobenius norm is held to u as well: independent roundings of at most u / sqrt(3) rms each.
"""
import math

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from qcache_util import D, ROW, codes_of, empty_cache, fractions_of, rows_of, values_of
from test_gpu_mixers import NAN, U, cu_of, gen_of, rand

pytestmark = pytest.mark.gpu
BITS = kb.KDA_DEVERR_CU_SEQLENS


def i64(x):
    return torch.tensor(list(x), dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------ append
def placed(cache, rows, lens_q, lens_k):
    want = cache.clone()
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        want[n, lk - lq:lk] = rows[a:a + lq]
        a += lq
    return want


@pytest.mark.parametrize("order", ["heads", "rows", "padded"])
@pytest.mark.parametrize("lens_q,lens_k,hk", [
    ([1], [1], 1), ([1, 1, 1], [9, 1, 40], 8), ([7, 0, 1, 300], [7, 5, 64, 301], 2), ([0, 0], [3, 0], 1), ([33] * 5, [33, 34, 40, 90, 50], 5),
    ([1] * 70, list(range(1, 71)), 4), ([2] + [0] * 1100 + [3], [2] + [4] * 1100 + [5], 1)])
def test_append_writes_the_exact_codes(lens_q, lens_k, hk, order):
    g = gen_of(sum(lens_k) + hk)
    T = sum(lens_q)
    k, v = rand(g, T + 2, hk, D, mul=3.0) + rand(g, hk, D, mul=2.0), rand(g, T + 2, 3 * hk * D)[:, hk * D:2 * hk * D].unflatten(1, (hk, D))
    cache = empty_cache(len(lens_q), max(lens_k) + 2, hk, order)
    want = placed(cache, rows_of(k[:T], v[:T]), lens_q, lens_k)
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    ko, vo = (torch.full((T + 2, hk, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    whole = torch.as_strided(cache, (cache.untyped_storage().nbytes(),), (1,), 0)
    gaps = whole.clone()
    torch.as_strided(gaps, cache.shape, cache.stride()).copy_(want)
    args = dict(cu_seqlens=cu_of(lens_q), status=status)
    kda.kda_qcache_append(k, v, cache, i64(lens_k), k_out=ko, v_out=vo, **args)
    assert kda.kda_read_device_status(status) == 0
    assert torch.equal(cache, want)
    assert torch.equal(whole, gaps)                                      # nothing between the rows either
    for x, xo in ((k, ko), (v, vo)):
        codes, scale, zero = codes_of(x[:T])
        ref = codes.double() * scale.double().repeat_interleave(64, -1) + zero.double().repeat_interleave(64, -1)
        assert ((xo[:T].double() - ref).abs() <= U * 1.0001 * ref.abs()).all()
        assert torch.isnan(xo[T:]).all()                                 # rows behind the last sequence
    # in place, and without the values
    k2, v2 = k.clone(), v.clone()
    kda.kda_qcache_append(k2, v2, cache.fill_(1), i64(lens_k), k_out=k2, v_out=v2, **args)
    assert torch.equal(k2[:T], ko[:T]) and torch.equal(v2[:T], vo[:T]) and torch.equal(k2[T:], k[T:]) and torch.equal(v2[T:], v[T:])
    again = empty_cache(len(lens_q), max(lens_k) + 2, hk, order)
    kda.kda_qcache_append(k, v, again, i64(lens_k), **args)
    assert torch.equal(again, want)
    if len(set(lens_q)) == 1:                                            # the same tokens a sequence: without cu_seqlens
        again = empty_cache(len(lens_q), max(lens_k) + 2, hk, order)
        kda.kda_qcache_append(k[:T], v[:T], again, i64(lens_k))
        assert torch.equal(again, want)


def special_vectors():
    """Vectors of 64 whose differences, quotients or ranges are hard."""
    g = torch.Generator().manual_seed(3)
    r = lambda: torch.randn(64, generator=g)
    out = [torch.zeros(64), torch.full((64,), -3.25), r() * 0, torch.cat([torch.zeros(32), -torch.zeros(32)])]
    out += [torch.arange(64).float() / 4, torch.arange(64).float() - 31, (torch.arange(64) % 31).float() / 2]        # ties
    for s in (1, 2, 3, 5, 7, 1.0078125, 1.9921875):                                                                 # every border itself
        x = torch.arange(64).float() % 31 / 2 * s
        x[0], x[1] = 0, 15 * s
        out += [x, x - 7.5 * s, -x]
    for lo in (-1.0, -7.5, -0.5, -96.0, -1.9921875):                       # numbers far below the range's precision, beside a border
        for tiny in (2.0 ** -20, 2.0 ** -60, 2.0 ** -126, 2.0 ** -133):
            x = r()
            x = x / x.abs().max() * abs(lo)
            x[:8] = torch.tensor([lo, -lo, 0.0, tiny, -tiny, 3 * tiny, -2.5 * tiny, lo / 2])
            x[8], x[9] = lo + 15.0, 0
            out.append(x)
    x = r()
    x[x < 0] *= 2.0 ** -40
    out += [x, -x, x.abs() + 2.0 ** -30, r() * 2.0 ** 60, r() * 2.0 ** -60, r() * 2.0 ** -122, r() * 2.0 ** -130, torch.full((64,), 2.0 ** -133)]
    big = torch.linspace(-1, 1, 64) * 3.38e38
    out += [big, big / 2, torch.cat([big[:1], r()[:62], big[-1:]])]        # a range that passes fp32's
    return torch.stack([x.bfloat16() for x in out])


def test_append_of_hard_numbers_is_exact():
    x = special_vectors()
    m = x.shape[0]
    k = torch.cat([x, x.flip(0)], 1)[:, None].cuda()
    v = torch.cat([x.roll(1, 0), x.flip(1)], 1)[:, None].cuda()
    cache = empty_cache(1, m, 1)
    kda.kda_qcache_append(k, v, cache, i64([m]))
    rows = cache[0, :, 0].cpu()
    numbers = rows[:, 128:].contiguous().view(torch.bfloat16)
    for i in range(m):
        for which, src in enumerate((k, v)):
            for half in range(2):
                codes, scale, zero = fractions_of(src[i, 0, 64 * half:64 * half + 64].cpu())
                at = 64 * which + 32 * half
                got = torch.stack([rows[i, at:at + 32] & 15, rows[i, at:at + 32] >> 4], -1).flatten().tolist()
                s, z = numbers[i, 4 * which + 2 * half:][:2]
                assert (float(s), float(z)) == (float(scale), float(zero)), (i, which, half)
                assert math.copysign(1, float(z)) == (-1 if zero < 0 else 1)
                assert got == codes, (i, which, half)


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_append_of_a_bad_value_reads_as_nan(bad):
    k, v = (rand(gen_of(5), 2, 1, D) for _ in "kv")
    k[0, 0, 70] = bad
    cache = empty_cache(1, 2, 1, fill=0)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kda.kda_qcache_append(k, v, cache, i64([2]), k_out=ko, v_out=vo)
    gk, gv = values_of(cache[0, :, 0])
    assert torch.isnan(gk[0, 64:]).all() and torch.isnan(ko[0, 0, 64:]).all()
    assert torch.isfinite(gk[0, :64]).all() and torch.isfinite(gk[1]).all() and torch.isfinite(gv).all() and torch.isfinite(vo).all()


@pytest.mark.parametrize("lens_q,lens_k,bad", [
    ([0, 2, 4], [3, 3], [0, 1][:0]), ([0, 2, 4], [9, 3], [0]), ([0, 2, 4], [3, 1], [1]), ([0, 2, 4], [-1, 4], [0]), ([0, 2, 9], [3, 8], [1]),
    ([1, 2, 4], [4, 4], [0]), ([0, -3, 4], [4, 8], [0, 1]), ([0, 1 << 40, 4], [4, 4], [0, 1]), ([0, 4, 2], [6, 6], [1]),
    ([0, 2, 4], [1 << 62, 4], [0]), ([0, 2, 4], [-(1 << 62), 4], [0]), ([0, 0, 4], [9, 4], [0]), ([0, 0, 4], [-1, 4], [0])])
def test_append_of_bad_lengths(lens_q, lens_k, bad):
    """Contents are checked on the device; a sequence that contradicts the tensors is left as it was."""
    g = gen_of(11)
    k, v = rand(g, 6, 2, D), rand(g, 6, 2, D)
    cache = empty_cache(2, 8, 2, fill=7)
    before = cache.clone()
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    kda.kda_qcache_append(k, v, cache, i64(lens_k), cu_seqlens=i64(lens_q), status=status)
    assert kda.kda_read_device_status(status) == (BITS if bad else 0)
    for n in range(2):
        if n in bad:
            assert torch.equal(cache[n], before[n])
        else:
            lq = lens_q[n + 1] - lens_q[n]
            want = before[n].clone()
            want[lens_k[n] - lq:lens_k[n]] = rows_of(k, v)[lens_q[n]:lens_q[n + 1]]
            assert torch.equal(cache[n], want)


def test_append_of_nothing():
    empty = torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    cache = empty_cache(2, 4, 2, fill=7)
    kda.kda_qcache_append(empty, empty, cache, i64([0, 4]), status=status)
    assert kda.kda_read_device_status(status) == 0 and (cache == 7).all()
    kda.kda_qcache_append(empty, empty, cache, i64([0, 5]), status=status)
    assert kda.kda_read_device_status(status) == BITS and (cache == 7).all()
    kda.kda_qcache_append(empty, empty, cache[:0], i64([]), status=status)               # no sequences
    kda.kda_qcache_append(empty, empty, cache[:, :0], i64([0, 0]))                       # no room


# ------------------------------------------------------------------ attention
def ref_attn(q, cache, scale, lens_q, lens_k):
    """(out, sum_j p_j |v_j|, sum_j p_j |v_j - w_j|, what rounded keys move, lse, largest sum of |q k|) over the packed
    queries, in 64 bits."""
    hq, hk = q.shape[1], cache.shape[2]
    shape = (sum(lens_q), hq, D)
    out, size, spread, moved = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(4))
    lse, most = torch.full(shape[:2], -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(shape[:2], dtype=torch.float64, device="cuda")
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        for h in range(hk):
            k, v = values_of(cache[n, :lk, h])
            g = slice(h * hq // hk, (h + 1) * hq // hk)
            qn = q[a:a + lq, g].double()
            w = torch.einsum("ihd,jd->hij", qn, k) * scale
            b = torch.einsum("ihd,jd->hij", qn.abs(), k.abs()) * scale
            seen = torch.arange(lk, device="cuda") <= torch.arange(lq, device="cuda")[:, None] + lk - lq
            w = w.masked_fill(~seen, -math.inf)
            l = torch.logsumexp(w, -1) if lk else torch.full(w.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
            p = torch.where(torch.isfinite(l)[..., None], (w - l[..., None]).exp(), 0.0)
            out[a:a + lq, g] = torch.einsum("hij,jd->ihd", p, v)
            size[a:a + lq, g] = torch.einsum("hij,jd->ihd", p, v.abs())
            spread[a:a + lq, g] = torch.einsum("hij,jd->ihd", p, (v - middles(cache[n, :lk, h])).abs())
            moved[a:a + lq, g] = torch.einsum("hij,jd->ihd", p * (b + (p * b).sum(-1, keepdim=True)), v.abs())
            lse[a:a + lq, g] = l.T
            if lk:
                most[a:a + lq, g] = (b * seen).amax(-1).T
        a += lq
    return out, size, spread, moved, lse, most


def middles(rows):
    """zero + 7.5 scale of the values' groups, for every channel."""
    numbers = rows[..., 136:].contiguous().view(torch.bfloat16).double()
    return (numbers[..., 1::2] + 7.5 * numbers[..., 0::2]).repeat_interleave(D // 2, -1)


def filled(g, lens_k, hk, order, room=None):
    """A cache whose rows past the lengths stand for NaN."""
    cache = empty_cache(len(lens_k), room or max(max(lens_k), 1) + 3, hk, order)
    mean = rand(g, hk, D, mul=0.5)
    for n, lk in enumerate(lens_k):
        cache[n, :lk] = rows_of(rand(g, lk, hk, D) + mean, rand(g, lk, hk, D) + 0.5 * mean)
    return cache


def check(got, lse, ref, many, total):
    out, size, spread, moved, rlse, most = ref
    got = got[:total].double()
    assert torch.isfinite(got).all()
    bound = 1.01 * (U * out.abs() + (2.0 ** -10 * size + U * U * moved if many else U * spread)) + 2.0 ** -14 * (size + spread + moved) + 1e-30
    over = (got - out).abs() - bound
    assert over.numel() == 0 or over.max().item() <= 0, f"{over.max().item():.3e} past its bound, {(over > 0).sum().item()} of {over.numel()}"
    if out.norm() > 0 and out.numel() > 4096:
        rel = ((got - out).norm() / out.norm()).item()
        assert rel <= U, rel
    if lse is not None:
        lse = lse[:total].double()
        empty = torch.isinf(rlse)
        assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
        tol = 2.0 ** -14 * (1 + most)
        assert ((lse - rlse).abs() <= tol)[~empty].all()


CASES = [
    # lens_q, lens_k, hq, hk, order
    ([1], [1], 1, 1, "heads"), ([1], [15], 4, 1, "rows"), ([1], [16], 8, 1, "heads"), ([1], [17], 8, 2, "padded"), ([1], [33], 5, 5, "heads"),
    ([1], [4097], 32, 8, "heads"), ([1] * 3, [0, 1, 64], 8, 2, "rows"), ([1] * 40, [(37 * i) % 700 for i in range(40)], 28, 4, "heads"),
    ([1] * 9, [2000, 1, 3, 0, 5000, 31, 32, 65, 100], 64, 8, "padded"), ([4] * 5, [4, 3, 900, 40, 0], 32, 8, "heads"),
    ([1, 8, 0, 3, 5], [1, 700, 90, 2, 64], 16, 2, "rows"), ([2, 3], [130, 257], 16, 1, "heads"), ([1, 1], [600, 601], 24, 1, "heads"),
    ([1], [700], 32, 1, "rows"), ([3, 1], [1200, 77], 40, 1, "padded"), ([1, 2], [300, 500], 128, 1, "heads"), ([1], [129], 96, 1, "heads"),
    ([0, 0, 1], [5, 0, 70], 4, 4, "heads"), ([17], [400], 4, 4, "heads"),
    # enough (sequence, head) units for two heads to go together
    ([1] * 40, [(53 * i) % 900 for i in range(40)], 28, 4, "rows"), ([2] * 20, [2 + (97 * i) % 800 for i in range(20)], 32, 8, "heads"),
    ([1] * 33, [5 * i for i in range(33)], 5, 5, "rows"), ([1] * 20, [300] * 20, 64, 8, "padded"), ([1] * 3 + [0] * 14 + [2] * 4, [4000] + [3] * 20, 32, 8, "rows"),
    # few rows on average, many in one sequence
    ([1] * 20 + [150], [40 * i for i in range(20)] + [700], 16, 2, "heads"),
    # prompts that continue: many rows
    ([100], [100], 8, 2, "heads"), ([1, 130, 300], [800, 130, 1300], 32, 8, "rows"), ([300], [200], 4, 1, "heads"), ([64, 65, 127, 1], [64, 200, 128, 1], 5, 5, "padded"),
    ([513], [1500], 16, 2, "heads"), ([40, 33], [2049, 33], 28, 4, "rows"), ([129, 2], [0, 500], 8, 1, "heads"), ([257], [640], 3, 1, "heads"), ([90], [333], 128, 1, "rows"),
]


def many_rows(T, n, cache, hq):
    """Whether a call's keys and values are expanded: by its tokens, sequences and the cache's room."""
    return T * (hq // cache.shape[2]) > 112 * n and T * hq * cache.shape[1] > 1 << 21


def wide(lens_q, hq):
    """Room for so many keys that many rows are taken as such."""
    return (1 << 21) // (sum(lens_q) * hq) + 1


# (those of many rows also with little room, where they are few)
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,order,more", [(*c, False) for c in CASES] +
                         [(*c, True) for c in CASES if sum(c[0]) * (c[2] // c[3]) > 112 * len(c[0])])
def test_attention(lens_q, lens_k, hq, hk, order, more):
    g = gen_of(sum(lens_k) + hq)
    T = sum(lens_q)
    cache = filled(g, lens_k, hk, order, room=max(wide(lens_q, hq), max(lens_k)) if more else None)
    q = rand(g, T + 3, (hq + 1) * D, mul=1.5)[:, D:].unflatten(1, (hq, D))
    out = torch.full((T + 3, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 3, hq), NAN, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    assert kda.kda_read_device_status(ws) == 0
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), many_rows(T + 3, len(lens_q), cache, hq), T)   # (the rows of q, those behind the last sequence among them)
    assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()     # rows behind the last sequence
    again, lse2 = torch.full_like(out, NAN), torch.full_like(lse, NAN)
    kda.kda_attn_qcache_fwd(q, cache, 0.1, again, i64(lens_k), lse=lse2, cu_seqlens_q=cu_of(lens_q), workspace=ws.fill_(255))
    assert torch.equal(again[:T], out[:T]) and torch.equal(lse2[:T], lse[:T])           # the same bits
    if len(set(lens_q)) == 1:
        again = torch.full_like(out, NAN)
        kda.kda_attn_qcache_fwd(q[:T], cache, 0.1, again[:T], i64(lens_k))               # without cu_seqlens_q and lse
        check(again, None, ref_attn(q, cache, 0.1, lens_q, lens_k), many_rows(T, len(lens_q), cache, hq), T)
        assert torch.isnan(again[T:]).all()


@pytest.mark.parametrize("lens_q,lens_k,hq,hk", [([1] * 6, [1, 40, 800, 3, 0, 96], 32, 8), ([60, 70], [500, 90], 16, 2)])
def test_attention_of_scores_that_matter(lens_q, lens_k, hq, hk):
    """Large scores, so that single keys win, scores far below them, and a scale of zero."""
    g = gen_of(77)
    cache = filled(g, lens_k, hk, "heads", room=1200)
    T = sum(lens_q)
    assert many_rows(T, len(lens_q), cache, hq) == (T > 100)
    q = rand(g, T, hq, D, mul=4.0)
    for scale in (0.0, 1e-6, 1.5):
        out = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, hq), NAN, device="cuda")
        kda.kda_attn_qcache_fwd(q, cache, scale, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
        if scale <= 1e-6:
            check(out, lse, ref_attn(q, cache, scale, lens_q, lens_k), many_rows(T, len(lens_q), cache, hq), T)
        else:       # scores in the hundreds: the weights' relative error is the scores' absolute one
            ref, size, spread, moved, rlse, most = ref_attn(q, cache, scale, lens_q, lens_k)
            unit = 2.0 ** -14
            err = (unit * most).clamp(max=40.0)[..., None]
            assert ((out.double() - ref).abs() <= U * (ref.abs() + size + spread) + 1.01 * (err.exp() - (-err).exp()) * largest(cache, lens_q, lens_k, hq) + 1e-30).all()


@pytest.mark.parametrize("lens_q,lens_k", [([2, 1], [300, 40]), ([90, 100], [500, 300])])
def test_attention_with_the_smallest_and_largest_scales(lens_q, lens_k):
    """A scale of 0 makes all keys alike, however large the products; one of 1e30 leaves a single key."""
    g = gen_of(78)
    hq, hk, T = 8, 2, sum(lens_q)
    cache = empty_cache(2, 1501, hk)
    assert many_rows(T, 2, cache, hq) == (T > 100)
    for power, scale in ((45, 0.0), (0, 1e30)):
        for n, lk in enumerate(lens_k):
            far = 2.0 ** -(torch.arange(lk, device="cuda") // 128 * 7 % 12).float()[:, None, None]   # (blocks of values, powers apart)
            cache[n, :lk] = rows_of(rand(g, lk, hk, D) * 2.0 ** power, (rand(g, lk, hk, D).float() * far).bfloat16())
        q = rand(g, T, hq, D) * 2.0 ** (power + 10 if power else 0)
        out, lse = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
        kda.kda_attn_qcache_fwd(q, cache, scale, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
        if scale == 0.0:
            check(out, lse, ref_attn(q, cache, scale, lens_q, lens_k), many_rows(T, len(lens_q), cache, hq), T)
            continue
        # a scale of 1e6 leaves the same single key where the first two scores are 1e-3 apart (weights of e^-1000)
        a = 0
        for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
            for h in range(hq):
                k, v = values_of(cache[n, :lk, h * hk // hq])
                w = q[a:a + lq, h].double() @ k.T
                w = w.masked_fill(torch.arange(lk, device="cuda") > torch.arange(lq, device="cuda")[:, None] + lk - lq, -math.inf)
                top = w.topk(2, -1)
                clear = top.values[:, 0] - top.values[:, 1] > 1e-3
                assert clear.float().mean() > 0.9
                got, want = out[a:a + lq, h].double(), v[top.indices[:, 0]]
                # the output's rounding, and a weight's (of less than the spread of its group, twice the row's largest)
                assert ((got - want).abs() <= 2.01 * U * (want.abs() + want.abs().amax(-1, keepdim=True)))[clear].all()
            a += lq


def largest(cache, lens_q, lens_k, hq):
    """The largest |v| that each query's channel can meet, [T, hq, 128]."""
    out = []
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        v = values_of(cache[n, :lk])[1].abs()
        top = v.amax(0) if lk else torch.zeros(cache.shape[2], D, dtype=torch.float64, device="cuda")
        out.append(top.repeat_interleave(hq // cache.shape[2], 0).expand(lq, hq, D))
    return torch.cat(out)


def test_attention_over_constant_groups_and_long_means():
    """Scales of zero, and keys and values whose mean is far larger than their spread."""
    g = gen_of(9)
    lens_k, hq, hk = [70, 1000], 8, 2
    k, v = rand(g, 1000, hk, D, mul=0.125) + 2.0, rand(g, 1000, hk, D, mul=0.0625) - 3.0
    k[::7, :, :64], v[::5, :, 64:] = 1.5, -0.75
    cache = empty_cache(2, 1001, hk)
    for n, lk in enumerate(lens_k):
        cache[n, :lk] = rows_of(k[:lk], v[:lk])
    q = rand(g, 2, hq, D)
    out, lse = torch.full((2, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((2, hq), NAN, device="cuda")
    kda.kda_attn_qcache_fwd(q, cache, 0.05, out, i64(lens_k), lse=lse)
    check(out, lse, ref_attn(q, cache, 0.05, [1, 1], lens_k), False, 2)


@pytest.mark.parametrize("tokens,hq,order", [(1, 16, "heads"), (1, 32, "rows"), (2, 64, "heads")])
def test_attention_of_many_short_sequences(tokens, hq, order):
    """Pieces of fewer slices than a CTA has warps, one after another: some warps have none and run ahead."""
    g = gen_of(41)
    hk, lens_k = 8, [2 + (37 * i) % 90 if i % 5 else 300 + i for i in range(600)]
    lens_q = [tokens] * len(lens_k)
    cache = filled(g, lens_k, hk, order)
    q = rand(g, sum(lens_q), hq, D)
    ref, first = ref_attn(q, cache, 0.08, lens_q, lens_k), None
    for _ in range(8):
        out, lse = torch.full_like(q, NAN), torch.full(q.shape[:2], NAN, device="cuda")
        kda.kda_attn_qcache_fwd(q, cache, 0.08, out, i64(lens_k), lse=lse)
        if first is None:
            check(out, lse, ref, False, q.shape[0])
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("lens_q,lens_k", [([3, 1, 2], [700, 300, 90]), ([70, 129, 65], [700, 300, 90])])
def test_attention_of_any_powers(lens_q, lens_k):
    """Queries and keys whose powers of two cancel, sequence by sequence; some rows and some blocks of keys far below the others."""
    g = gen_of(31)
    hq, hk, T = 8, 2, sum(lens_q)
    cache, q = empty_cache(len(lens_k), 1101, hk), rand(g, T, hq, D)
    many = many_rows(T, 3, cache, hq)
    assert many == (T > 100)
    a = 0
    for n, (lq, lk, power) in enumerate(zip(lens_q, lens_k, (40, -45, 0))):
        small = torch.ones(lk, 1, 1, device="cuda")
        small[200:380], small[5::9] = 2.0 ** -9, 2.0 ** -30
        k = rand(g, lk, hk, D).float() * small * 2.0 ** -power
        cache[n, :lk] = rows_of(k.bfloat16(), rand(g, lk, hk, D) * 2.0 ** (power // 2))
        few = torch.ones(lq, 1, 1, device="cuda")
        few[1::3], few[2::7] = 2.0 ** -12, 0.0
        q[a:a + lq] = (q[a:a + lq].float() * few * 2.0 ** power).bfloat16()
        q[a:a + lq, :, 3] *= 2.0 ** -20
        a += lq
    out, lse = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hq), NAN, device="cuda")
    kda.kda_attn_qcache_fwd(q, cache, 0.09, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    ref = ref_attn(q, cache, 0.09, lens_q, lens_k)
    for r in zip(lens_q, [sum(lens_q[:n]) for n in range(3)]):   # (a sequence by itself: their values differ by powers of two)
        rows = slice(r[1], sum(r))
        check(out[rows], lse[rows], [x[rows] for x in ref], many, r[0])


@pytest.mark.parametrize("lens_q,lens_k", [
    ([0, 1, 2], [3, 9]), ([0, 1, 2], [-1, 3]), ([0, 1, 9], [3, 3]), ([1, 1, 2], [3, 3]), ([0, 3, 2], [3, 3]), ([0, 1, 2], [1 << 40, 3]),
    ([0, -1, 2], [3, 3]), ([0, 1 << 40, 2], [3, 3]), (None, [3, 9]), (None, [-5, 3])])
def test_attention_of_bad_lengths(lens_q, lens_k):
    g = gen_of(12)
    cache = filled(g, [8, 8], 2, "heads", room=8)
    for tokens in (2, 200):
        q = rand(g, tokens, 4, D)
        out = torch.full((tokens, 4, D), NAN, dtype=torch.bfloat16, device="cuda")
        if lens_q and max(lens_q) == 9 and tokens > 2:
            continue
        ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), cu_seqlens_q=None if lens_q is None else i64(lens_q))
        assert kda.kda_read_device_status(ws) == BITS
        assert torch.isnan(out).all()


def test_attention_of_nothing():
    g = gen_of(13)
    cache = filled(g, [4, 0], 2, "heads")
    empty = torch.empty(0, 4, D, dtype=torch.bfloat16, device="cuda")
    kda.kda_attn_qcache_fwd(empty, cache, 0.1, empty.clone(), i64([4, 0]))                        # no queries
    q, out = rand(g, 2, 4, D), torch.full((2, 4, D), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 4), NAN, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache[:, :0], 0.1, out, i64([0, 0]), lse=lse)                 # a cache without room
    assert kda.kda_read_device_status(ws) == 0 and (out == 0).all() and (lse == -math.inf).all()
    kda.kda_attn_qcache_fwd(empty, cache[:0], 0.1, empty.clone(), i64([]))                        # no sequences
    kda.kda_attn_qcache_fwd(q, cache[:0], 0.1, out.fill_(NAN), i64([]), cu_seqlens_q=i64([0]))
    assert torch.isnan(out).all()


@pytest.mark.parametrize("T,lens_k,hq", [(3, [900, 33, 5000], 32), (400, [900, 700, 5000], 8)])
def test_captured_and_replayed(T, lens_k, hq):
    """Append and attention in one graph; a replay takes new tokens and lengths, and other graphs may share the workspace."""
    g = gen_of(21)
    n, hk = len(lens_k), 4
    per = [1, 1, 1] if T == 3 else [200, 150, 50]
    cache = filled(g, lens_k, hk, "heads", room=5600)
    k, v, q = rand(g, T, hk, D), rand(g, T, hk, D), rand(g, T, hq, D)
    lens, cu = i64(lens_k), cu_of(per)
    out = torch.zeros_like(q)
    ws = torch.empty(kda.kda_attn_qcache_workspace_size(T, hq, hk, n, 5600), dtype=torch.uint8, device="cuda")

    def both(o):
        kda.kda_qcache_append(k, v, cache, lens, cu_seqlens=cu)
        kda.kda_attn_qcache_fwd(q, cache, 0.1, o, lens, cu_seqlens_q=cu, workspace=ws)

    both(out)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(out)
        graphs.append(graph)
    for step in range(3):
        lens += i64(per)
        for t in (k, v, q):
            t.copy_(rand(g, *t.shape))
        graphs[step % 2].replay()
        got, rows = out.clone(), cache.clone()
        assert kda.kda_read_device_status(ws) == 0
        out.zero_()
        both(out)
        assert torch.equal(got, out) and torch.equal(rows, cache)
        lens_k = [a + b for a, b in zip(lens_k, per)]
        check(got, None, ref_attn(q, cache, 0.1, per, lens_k), many_rows(T, n, cache, hq), T)


@pytest.mark.parametrize("lens_q,lens_k,hq", [([1] * 6, [900, 33, 5000, 1, 0, 64], 32), ([200, 40], [900, 40], 8)])
def test_two_at_once(lens_q, lens_k, hq):
    """Calls that overlap on two streams, each with its own workspace and inputs."""
    g = gen_of(24)
    T, hk = sum(lens_q), 4
    sides = []
    for _ in range(2):
        cache, q = filled(g, lens_k, hk, "heads", room=5003), rand(g, T, hq, D)
        assert many_rows(T, len(lens_q), cache, hq) == (T > 100)
        want = torch.empty_like(q)
        kda.kda_attn_qcache_fwd(q, cache, 0.1, want, i64(lens_k), cu_seqlens_q=cu_of(lens_q))
        sides.append((torch.cuda.Stream(), cache, q, want, torch.empty_like(q), i64(lens_k), cu_of(lens_q)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, cache, q, want, out, lens, cu in sides:
            kda.kda_attn_qcache_fwd(q, cache, 0.1, out, lens, cu_seqlens_q=cu, stream=s)
    torch.cuda.synchronize()
    for s, cache, q, want, out, lens, cu in sides:
        assert torch.equal(out, want)


def test_many_rows_with_key_heads_in_several_turns():
    """Room for so many keys that the expanded ones fit into the workspace for three of the eight key heads at a time only."""
    g = gen_of(25)
    n, hk, hq, room, lens_q, lens_k = 2, 8, 16, 260_000, [90, 60], [700, 200]
    cache = empty_cache(n, room, hk)
    for i, lk in enumerate(lens_k):
        cache[i, :lk] = rows_of(rand(g, lk, hk, D), rand(g, lk, hk, D))
    T = sum(lens_q)
    assert T * (hq // hk) > 128 * n
    q, lse = rand(g, T, hq, D), torch.full((T, hq), NAN, device="cuda")
    out = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse, cu_seqlens_q=cu_of(lens_q))
    assert kda.kda_read_device_status(ws) == 0 and ws.numel() < 1.1 * 2 ** 30
    check(out, lse, ref_attn(q, cache, 0.1, lens_q, lens_k), True, T)
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out.fill_(NAN), i64([room + 1, 3]), cu_seqlens_q=cu_of(lens_q), workspace=ws)
    assert kda.kda_read_device_status(ws) == BITS and torch.isnan(out).all()


def test_on_another_stream():
    g = gen_of(22)
    lens_k = [900, 33, 5000]
    cache, q = filled(g, lens_k, 4, "heads"), rand(g, 3, 16, D)
    want, out = torch.empty_like(q), torch.empty_like(q)
    lens = i64(lens_k)
    kda.kda_attn_qcache_fwd(q, cache, 0.1, want, lens)
    torch.cuda.synchronize()
    for how in ("stream", "handle"):
        s = torch.cuda.Stream()
        out.zero_()
        torch.cuda.synchronize()
        ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, lens, stream=s if how == "stream" else s.cuda_stream)
        assert kda.kda_read_device_status(ws, stream=s) == 0 and torch.equal(out, want)


def test_workspaces_are_kept_only_when_nobody_holds_them():
    g = gen_of(26)
    lens_k = [900, 33, 5000]
    cache, q, lens = filled(g, lens_k, 4, "heads"), rand(g, 3, 16, D), i64(lens_k)
    out = torch.empty_like(q)
    call = lambda **kw: kda.kda_attn_qcache_fwd(q, cache, 0.1, out, lens, **kw)
    at = call().data_ptr()
    assert call().data_ptr() == at                                   # dropped: taken again
    held = call()
    second = call()
    assert second.data_ptr() != held.data_ptr()
    view, ptr = second[:4], second.data_ptr()
    del second
    assert call().data_ptr() != ptr                                  # a view keeps it too
    third = call()
    storage, ptr = third.untyped_storage(), third.data_ptr()
    del third
    assert call().data_ptr() != ptr and storage.data_ptr() == ptr    # ... and its storage
    bad = i64([1 << 40, 1, 1])
    first = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, bad)
    call()
    assert kda.kda_read_device_status(first) == BITS                 # a later call does not overwrite a status that is held
    assert kda.kda_read_device_status(view) == 0
    mine = call().data_ptr()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = call().data_ptr()
        assert call().data_ptr() == other != mine                    # a stream's own
    torch.cuda.synchronize()
    assert call(stream=s).data_ptr() not in (mine, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call().data_ptr()
    assert captured not in (mine, other)
    want = out.clone()
    graph.replay()
    assert torch.equal(out, want)


def test_a_cache_past_32_bits():
    """Rows whose byte offsets pass 2^32, in both the sequence and the row direction."""
    g = gen_of(23)
    n, hk, room = 3, 2, 5_400_000                                          # 4.67 GB, 1.56 GB a sequence
    cache = torch.zeros(n, hk, room, ROW, dtype=torch.uint8, device="cuda").transpose(1, 2)
    k, v, q = rand(g, 3 * 40, hk, D), rand(g, 3 * 40, hk, D), rand(g, 3, 8, D)
    per = [40, 40, 40]
    lens_k = [room, 40, room - 1]
    kda.kda_qcache_append(k, v, cache, i64(lens_k), cu_seqlens=cu_of(per))
    want = rows_of(k, v)
    assert torch.equal(cache[2, room - 41:room - 1], want[80:]) and torch.equal(cache[0, room - 40:], want[:40]) and torch.equal(cache[1, :40], want[40:80])
    assert (cache[2, room - 45:room - 41] == 0).all()
    # zeros stand for keys and values of zero: their weights are exp(0) each
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    ws = kda.kda_attn_qcache_fwd(q, cache, 0.1, out, i64(lens_k), lse=lse)
    assert kda.kda_read_device_status(ws) == 0
    for i in range(3):
        kk, vv = (x.repeat_interleave(4, 1) for x in values_of(want[40 * i:40 * i + 40]))
        w = torch.einsum("hd,jhd->hj", q[i].double(), kk) * 0.1
        zeros = lens_k[i] - 40
        l = torch.logsumexp(torch.cat([w, torch.full((8, 1), math.log(zeros) if zeros else -math.inf, device="cuda", dtype=torch.float64)], 1), -1)
        ref = torch.einsum("hj,jhd->hd", (w - l[:, None]).exp(), vv)
        p = (w - l[:, None]).exp()
        size = torch.einsum("hj,jhd->hd", p, vv.abs())
        spread = torch.einsum("hj,jhd->hd", p, (vv - middles(want[40 * i:40 * i + 40]).repeat_interleave(4, 1)).abs())
        assert ((out[i].double() - ref).abs() <= U * (ref.abs() + spread) + 2.0 ** -13 * (size + spread)).all()
        assert ((lse[i].double() - l).abs() <= 2.0 ** -12).all()
