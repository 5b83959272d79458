"""The token mixers beside KDA on the GPU: how batches are divided among the SMs, graphs, and values
that are not finite.  The bounds are those of test_gpu_mixers.py.
"""
import random

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import D, NAN, check_attn, check_lin_out, check_state, cu_of, gen_of, rand, ref_attn, ref_lin

pytestmark = pytest.mark.gpu


def attn_packed(seed, lens, hq, hk, lens_k=None):
    g = gen_of(seed)
    lens_k = lens if lens_k is None else lens_k
    q, k, v = rand(g, sum(lens), hq, D), rand(g, sum(lens_k), hk, D), rand(g, sum(lens_k), hk, D)
    out = torch.full_like(q, NAN)
    lse = torch.full((sum(lens), hq), NAN, device="cuda")
    ws = kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, cu_seqlens_q=cu_of(lens), cu_seqlens_k=cu_of(lens_k))
    assert kda.kda_read_device_status(ws) == 0
    at = [0] + torch.tensor(lens_k).cumsum(0).tolist()
    check_attn(q, out, lse, ref_attn(q, k, v, 0.1, lens, lens_k, lambda n: (k[at[n]:at[n + 1]], v[at[n]:at[n + 1]])), 0.1)


@pytest.mark.parametrize("nseq,hq,hk", [(383, 2, 1), (385, 4, 2), (1000, 2, 2)])
def test_attn_more_sequences_than_threads(nseq, hq, hk):
    r = random.Random(nseq)
    attn_packed(nseq, [r.choice([0, 1, 1, 2, 5, 33]) for _ in range(nseq)], hq, hk)


@pytest.mark.parametrize("hq,hk", [(8, 2), (32, 8), (20, 1)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attn_shares_of_one_tile_and_two_tile_pairs(hq, hk, seed):
    """Ragged lengths around a tile's tokens: pairs with one tile and with two take turns in a share."""
    r, tq = random.Random(seed), 128 * hk // hq
    lens = [max(0, r.choice([1, tq, 2 * tq, 3 * tq, 7 * tq]) + r.randint(-3, 3)) for _ in range(40)]
    attn_packed(seed, lens, hq, hk, [n + r.choice([0, 0, 1, 127, 128, 500]) for n in lens])


@pytest.mark.parametrize("hq,hk,lens_k", [(8, 8, [30000]), (8, 1, [20000, 1, 9000]), (128, 1, [6000])])
def test_attn_single_tokens_over_many_shares(hq, hk, lens_k):
    g = gen_of(hq)
    n, room = len(lens_k), max(lens_k)
    q, k, v = rand(g, n, hq, D, mul=3.0), rand(g, n, room, hk, D), rand(g, n, room, hk, D)
    out, lse = torch.full_like(q, NAN), torch.full((n, hq), NAN, device="cuda")
    ws = kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, seqlens_k=torch.tensor(lens_k, device="cuda"))
    assert kda.kda_read_device_status(ws) == 0
    check_attn(q, out, lse, ref_attn(q, k, v, 0.1, [1] * n, lens_k, lambda i: (k[i, :lens_k[i]], v[i, :lens_k[i]])), 0.1)


@pytest.mark.parametrize("lens", [[40, 200], [2200]], ids=["whole", "split"])
def test_attn_nan_stays_in_its_row_and_heads(lens):
    g = gen_of(9)
    T = sum(lens)
    q, k, v = rand(g, T, 4, D), rand(g, T, 2, D), rand(g, T, 2, D)
    clean, out = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    lse = torch.full((T, 4), 5.0, device="cuda")
    kda.kda_attn_fwd(q, k, v, 0.1, clean, cu_seqlens_q=cu_of(lens))
    row = T - 5                                            # a late query: its pair is cut in the long prompt
    q[row, 1, 3] = NAN
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, cu_seqlens_q=cu_of(lens))
    assert torch.isnan(out[row, 1]).all() and torch.isnan(lse[row, 1])
    out[row, 1] = clean[row, 1]
    assert torch.equal(out, clean)
    lse[row, 1] = 0.0
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("nseq,h", [(767, 1), (769, 2), (1600, 1)])
def test_lin_more_sequences_than_threads(nseq, h):
    r = random.Random(nseq)
    lens = [r.choice([0, 1, 1, 2]) for _ in range(nseq)]
    lens[nseq // 3], lens[-2] = 300, 130
    g = gen_of(nseq)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld = torch.full((h,), -0.05, device="cuda")
    init, final = rand(g, nseq, h, D, D), torch.full((nseq, h, D, D), NAN, device="cuda")
    out = torch.full_like(q, NAN)
    ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
    assert kda.kda_read_device_status(ws) == 0
    o, A, s, t = ref_lin(q[0], k[0], v[0], ld, 0.1, lens, init)
    check_lin_out(out[0], o, A)
    check_state("final_state", final, s, t)


def test_lin_units_over_many_shares_beside_short_ones():
    """One head of a prompt of 60 chunks among short prompts: units in many, in two and in one share;
    the same bits again, and the state against 64 bits (the recurrence in closed form)."""
    lens, h = [130, 7680, 5, 900], 2
    g = gen_of(31)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld = torch.tensor([-0.001, -0.5], device="cuda")
    init = rand(g, len(lens), h, D, D, dtype=torch.float32)
    res = []
    for _ in range(3):
        out, final = torch.full_like(q, NAN), torch.full((len(lens), h, D, D), NAN, device="cuda")
        ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
        assert kda.kda_read_device_status(ws) == 0
        res.append((out, final))
    assert all(torch.equal(a, b) for r in res[1:] for a, b in zip(r, res[0]))
    a = 0
    for n, L in enumerate(lens):
        w = torch.exp(ld.double()[:, None] * torch.arange(L - 1, -1, -1, device="cuda"))          # [h, L]
        vw, kk = v[0, a:a + L].double().transpose(0, 1) * w[..., None], k[0, a:a + L].double().transpose(0, 1)
        f = torch.exp(ld.double() * L)[:, None, None]
        s = f * init[n].double() + vw.transpose(1, 2) @ kk
        t = f * init[n].double().abs() + vw.abs().transpose(1, 2) @ kk.abs()
        check_state("final_state", final[n], s, t)
        a += L


def chunked_lin(q, k, v, ld, scale, lens, init):
    """ref_lin of test_gpu_mixers.py with the recurrence unrolled over 64 tokens at a time."""
    outs, bounds, finals, finals_abs, a = [], [], [], [], 0
    d = ld.double()[:, None]
    for n, L in enumerate(lens):
        s = init[n].double()
        t = s.abs()
        for c in range(a, a + L, 64):
            m = min(64, a + L - c)
            i = torch.arange(m, device="cuda")
            qc, kc, vc = (x[c:c + m].double().transpose(0, 1) for x in (q, k, v))
            low = torch.exp(d[..., None] * (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
            into, w, f = torch.exp(d * (i + 1))[..., None], torch.exp(d * (m - 1 - i))[..., None], torch.exp(d * m)[..., None]
            outs.append(scale * ((qc @ kc.mT * low) @ vc + into * (qc @ s.mT)).transpose(0, 1))
            bounds.append(scale * ((qc.abs() @ kc.abs().mT * low) @ vc.abs() + into * (qc.abs() @ t.mT)).transpose(0, 1))
            s = f * s + (vc * w).mT @ kc
            t = f * t + (vc * w).abs().mT @ kc.abs()
        a += L
        finals.append(s)
        finals_abs.append(t)
    return torch.cat(outs), torch.cat(bounds), torch.stack(finals), torch.stack(finals_abs)


DIVIDED = [([94, 1407], 64), ([2018, 3165, 32], 40), ([18, 2659, 278, 2, 260], 48), ([1212, 3, 4993], 16), ([2738, 6000], 8), ([5000], 5)]
for _seed in range(10):
    _r = random.Random(_seed)
    DIVIDED.append(([int(2 ** _r.uniform(0, 12)) for _ in range(_r.randint(1, 7))], _r.choice([1, 3, 7, 16, 30, 64])))


@pytest.mark.parametrize("lens,h", DIVIDED, ids=[f"{'-'.join(map(str, a))}x{b}" for a, b in DIVIDED])
def test_lin_however_the_units_are_divided(lens, h):
    """Shares that end one unit, hold others and begin a third, each of them in one, two or more shares."""
    g = gen_of(sum(lens) + h)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld = -(2.0 ** (-10.0 * torch.arange(1, h + 1) / h)).cuda()
    init, final = rand(g, len(lens), h, D, D, dtype=torch.float32), torch.full((len(lens), h, D, D), NAN, device="cuda")
    out = torch.full_like(q, NAN)
    ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
    assert kda.kda_read_device_status(ws) == 0
    o, A, s, t = chunked_lin(q[0], k[0], v[0], ld, 0.1, lens, init)
    check_lin_out(out[0], o, A)
    check_state("final_state", final, s, t)


def test_mixers_in_a_graph():
    """One capture of all four, replayed on new inputs: the bits of plain calls."""
    hq, hk, lens, S = 8, 2, [150, 61, 700], 600
    T, n, reach = sum(lens), len(lens), 1024
    g = gen_of(41)
    angle = torch.arange(reach, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    cu = cu_of(lens)
    pos = torch.cat([torch.arange(x) for x in lens]).cuda()
    lens_k = torch.tensor([1, 600, 333], device="cuda")
    q, k, v = rand(g, T, hq, D), rand(g, T, hk, D), rand(g, T, hk, D)
    w = rand(g, D, dtype=torch.float32)
    kc, vc = rand(g, n, S, hk, D), rand(g, n, S, hk, D)
    lq, lk, lv = (rand(g, 1, T, hq, D) for _ in range(3))
    sq, sk, sv = (rand(g, n, hq, D) for _ in range(3))
    ld = torch.full((hq,), -0.1, device="cuda")
    res = {name: torch.empty_like(x) for name, x in dict(q=q, k=k, o=q, step=q[:n], lin=lq, lstep=sq).items()}
    state = torch.empty(n, hq, D, D, device="cuda")

    def work(r, state):
        kda.kda_qk_norm_rope(q, k, w, w, cs, pos, r["q"], r["k"])
        kda.kda_attn_fwd(r["q"], r["k"], v, 0.1, r["o"], cu_seqlens_q=cu)
        kda.kda_attn_fwd(r["q"][:n], kc, vc, 0.1, r["step"], seqlens_k=lens_k)
        kda.kda_lin_fwd(lq, lk, lv, ld, 0.1, r["lin"], final_state=state, cu_seqlens=cu)
        kda.kda_lin_decode(sq, sk, sv, ld, 0.1, r["lstep"], initial_state=state, final_state=state)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(res, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(res, state)
    for round_ in range(2):
        for x in (q, k, v, lq, lk, lv, sq, sk, sv):
            x.copy_(rand(g, *x.shape))
        for x in res.values():
            x.fill_(NAN)
        graph.replay()
        plain, plain_state = {a: torch.full_like(b, NAN) for a, b in res.items()}, torch.empty_like(state)
        work(plain, plain_state)
        torch.cuda.synchronize()
        for a in res:
            assert torch.equal(res[a], plain[a]), a
        assert torch.equal(state, plain_state)
