"""The operators around the mixers in runs of them, as a model uses them."""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb
from qcache_util import empty_cache, values_of
from test_gpu_example import load_example
from test_gpu_mixers import D, NAN, U, cu_of, gen_of, rand, table
from test_gpu_qcache import check, i64, ref_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,steps", [((37, 1, 200, 130), 5), ((5,), 2), ((300, 64, 129, 31, 1, 90), 1)])
def test_example_with_its_cache_in_4_bits(lens, steps):
    # as without: three layers round to bf16 five times on their way (norm, projection, mixer, gate, product), by at most
    # 2^-8 each and independently between the two runs.  The cache adds nothing of its own where both runs put the
    # same codes into it; a key or value that differs in its last bit between them (by at most 2 * 2^-8 of itself) moves
    # to a neighbouring code, a fifteenth of its group's range and so at most about 2 / 15 of the
    # group's largest number, where it lay within that of a border: a share of 2 * 2^-8 * 7.5 of the numbers at
    # most, each off by (2 / 15), in the root mean square sqrt(15 * 2^-8) * 2 / 15 = 0.032 of the largest, a third of that of
    # the group's own size (64 numbers): 0.097
    assert load_example().check(lens, steps, cache4=True) <= 2 ** 0.5 * 15 * 2.0 ** -8 + 0.097


def test_decode_steps_of_a_layer_over_a_cache_in_4_bits():
    """residual norm, projection, norm and rotation, append, attention, projection, some steps long in one graph."""
    g = gen_of(41)
    n, hidden, hq, hk, room = 5, 512, 8, 2, 96
    lens_k = [0, 3, 17, 64, 80]
    w_in, w_out = rand(g, hidden, (hq + 2 * hk) * D, mul=hidden ** -0.5), rand(g, hq * D, hidden, mul=(hq * D) ** -0.5)
    weight, cs = 1 + rand(g, hidden, mul=0.1, dtype=torch.float32), table(128, 64)
    cache = empty_cache(n, room, hk)
    old = rand(g, sum(lens_k), hk, D), rand(g, sum(lens_k), hk, D)
    kda.kda_qcache_append(*old, cache, i64(lens_k), cu_seqlens=cu_of(lens_k))
    stream, lens, last = rand(g, n, hidden, dtype=torch.float32), i64(lens_k), rand(g, n, hidden)
    normed, out = torch.empty(n, hidden, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hq, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.kda_attn_qcache_workspace_size(n, hq, hk, n, room), dtype=torch.uint8, device="cuda")
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    qkv = torch.empty(n, (hq + 2 * hk) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([hq * D, hk * D, hk * D], 1))

    def step():
        kda.kda_residual_norm(last, stream, weight, normed, residual_out=stream, scale=0.5)
        torch.matmul(normed, w_in, out=qkv)
        kda.kda_qk_norm_rope(q, k, None, None, cs, lens, q, k)
        lens.add_(1)
        kda.kda_qcache_append(k, v, cache, lens, status=status)
        kda.kda_attn_qcache_fwd(q, cache, D ** -0.5, out, lens, workspace=ws)
        torch.matmul(out.flatten(1), w_out, out=last)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = [t.clone() for t in (stream, lens, last, cache)]
    with torch.cuda.stream(side):
        step()                                     # (warms the products up)
    torch.cuda.current_stream().wait_stream(side)
    for t, was in zip((stream, lens, last, cache), kept):
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        before, was = stream.clone(), last.clone()
        graph.replay()
        lens_k = [a + 1 for a in lens_k]
        assert lens.tolist() == lens_k
        assert kda.kda_read_device_status(ws) == 0 and kda.kda_read_device_status(status) == 0
        want = before.double() + 0.5 * was.double()
        assert ((stream.double() - want).abs() <= 2.0 ** -22 * (before.abs() + was.abs())).all()
        check(out, None, ref_attn(q, cache, D ** -0.5, [1] * n, lens_k), False, n)
        for s in range(n):                         # the new row stands for this step's key and value, within half a step of the codes
            for x, y in zip((k[s], v[s]), values_of(cache[s, lens_k[s] - 1])):
                r = x.double().unflatten(-1, (2, 64))
                half = (r.amax(-1) - r.amin(-1)) / 15 * (0.5 + 15 * 2.0 ** -8)
                assert ((y.unflatten(-1, (2, 64)) - r).abs() <= half[..., None]).all()
    bad = lens.clone().fill_(room)
    lens.copy_(bad)                                # no room for another token: nothing is written, the bits say so
    rows = cache.clone()
    graph.replay()
    assert kda.kda_read_device_status(ws) == kda.kda_read_device_status(status) == kb.KDA_DEVERR_CU_SEQLENS
    assert torch.equal(rows, cache)


def test_prompts_see_what_later_steps_see():
    """Attention over the appended values themselves, and later over the cache, answers the same query the same way."""
    g = gen_of(42)
    lens, hq, hk = [150, 33, 1], 8, 2
    T = sum(lens)
    q, k, v = rand(g, T, hq, D), rand(g, T, hk, D), rand(g, T, hk, D)
    cache = empty_cache(3, 160, hk, "rows")
    kda.kda_qcache_append(k, v, cache, i64(lens), cu_seqlens=cu_of(lens), k_out=k, v_out=v)
    a, b = (torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    kda.kda_attn_fwd(q, k, v, D ** -0.5, a, cu_seqlens_q=cu_of(lens))
    kda.kda_attn_qcache_fwd(q, cache, D ** -0.5, b, i64(lens), cu_seqlens_q=cu_of(lens))
    out, size, spread, moved, _, _ = ref_attn(q, cache, D ** -0.5, lens, lens)
    # the appended values are rounded once more (keys and values, as far as the last term), the weights and results of each too
    assert ((a.double() - b.double()).abs() <= U * 1.01 * (2 * out.abs() + 2 * size + spread + moved) + 2.0 ** -14 * (size + moved)).all()
