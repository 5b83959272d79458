"""The token mixers beside KDA on the GPU, against plain evaluations of their formulas in 64 bits.

Bounds, per element, with u = 2^-8 the unit roundoff of bf16 (8 significant bits):
  norm_rope   u |y| for the output's rounding, 2^-18 (|a| + |b|) for the fp32 arithmetic
  attention   u |o| + u sum_j p_j |v_j| (the weights rounded to bf16 for the product with v)
  linear      u |o| + u A, A = scale sum_j a^(i-j) sum_k |q_k k_jk| |v_j| + the initial state's part, which
              bounds the error of rounding the scores and the carried state; and, since the errors
              are independent, 2^-8 in the Frobenius norm
  states      2^-17 of the recurrence over absolute values (a chunk's sums in fp32, up to 64
              truncating additions of 2^-23)
The inputs that a mask excludes hold NaN where the interface promises not to use them.
"""
import math

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from gated_delta_rule_36_gb300 import binding as kb

pytestmark = pytest.mark.gpu
D = 128
U = 2.0 ** -8
NAN = float("nan")


def rand(gen, *shape, mul=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * mul).to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cu_of(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0).cuda()


def within(name, got, ref, bound):
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    over = (got - ref).abs() - bound
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{name}: an element is {worst:.3e} past its bound ({(over > 0).sum().item()} of {over.numel()})"


# ---------------------------------------------------------------- norm and rotation
def table(reach, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(reach, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def ref_rope(x, w, cs, pos, eps, interleaved):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w.double())
    bound = U * 1.01 * y.abs() + 2.0 ** -18 * y.abs()
    if cs is not None:
        half = cs.shape[1] // 2
        c, s = (t[:, None] for t in cs.double()[pos].split(half, 1))
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ya, yb = y[..., a], y[..., b]
        y = y.clone()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        bound = U * 1.01 * y.abs()
        bound[..., a] += 2.0 ** -18 * (ya.abs() + yb.abs())
        bound[..., b] += 2.0 ** -18 * (ya.abs() + yb.abs())
        bound += 2.0 ** -18 * y.abs()
    return y, bound


@pytest.mark.parametrize("T,hq,hk,rot,inter,weighted,fused", [
    (1, 1, 1, 128, False, True, False), (7, 5, 5, 64, False, True, True), (33, 28, 4, 128, True, True, True),
    (129, 8, 1, 16, True, False, False), (1000, 32, 8, 96, False, True, True), (64, 40, 8, 0, False, True, True),
    (5, 64, 8, 112, False, False, False), (300, 3, 1, 32, False, True, False)])
def test_norm_rope(T, hq, hk, rot, inter, weighted, fused):
    g = gen_of(T + hq)
    if fused:
        qkv = rand(g, T, (hq + 2 * hk) * D, mul=3.0)
        q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    else:
        q, k = rand(g, T, hq, D, mul=0.01), rand(g, T, hk, D, mul=30.0)
    q[T // 2] = 0.0                                     # a row of zeros: the norm is eps
    wq, wk = (rand(g, D, dtype=torch.float32), rand(g, D, dtype=torch.float32)) if weighted else (None, None)
    cs = table(5000, rot) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda") if rot else None
    qo, ko = torch.full((T, hq, D), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((T, hk, D), NAN, dtype=torch.bfloat16, device="cuda")
    before = q.clone(), k.clone()
    kda.kda_qk_norm_rope(q, k, wq, wk, cs, pos, qo, ko, flags=kda.KDA_FLAG_ROPE_INTERLEAVED if inter else 0)
    for name, x, w, y in (("q", q, wq, qo), ("k", k, wk, ko)):
        ref, bound = ref_rope(x, w, cs, pos, 1e-6, inter)
        within(name, y, ref, bound)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    kda.kda_qk_norm_rope(q, k, wq, wk, cs, pos, q, k, flags=kda.KDA_FLAG_ROPE_INTERLEAVED if inter else 0)   # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_norm_rope_without_keys_and_positions_outside_the_table():
    g = gen_of(1)
    T, h = 9, 3
    q, cs = rand(g, T, h, D), table(50, 64)
    pos = torch.tensor([0, 49, 50, -1, 7, 1 << 40, 3, 3, 3], device="cuda")
    bad = torch.tensor([2, 3, 5], device="cuda")
    out = torch.empty_like(q)
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    kda.kda_qk_norm_rope(q, None, None, None, cs, pos, out, None, status=status)
    assert kda.kda_read_device_status(status) == kb.KDA_DEVERR_POSITION
    assert torch.isnan(out[bad]).all()
    good = [i for i in range(T) if i not in (2, 3, 5)]
    ref, bound = ref_rope(q[good], None, cs, pos[good], 1e-6, False)
    within("q", out[good], ref, bound)
    kda.kda_qk_norm_rope(q[:0], None, None, None, cs, pos[:0], out[:0], None)     # no tokens: nothing to do
    empty = torch.empty(0, 64, device="cuda")
    kda.kda_qk_norm_rope(q, None, None, None, empty, pos, out, None)              # an empty table: every position is outside
    assert torch.isnan(out).all()


# ---------------------------------------------------------------- attention
def ref_attn(q, k, v, scale, lens_q, lens_k, kv_of):
    """(out, bound, lse) over the packed queries; kv_of(n) gives sequence n's keys and values."""
    hq = q.shape[1]
    out = torch.zeros(sum(lens_q), hq, D, dtype=torch.float64, device="cuda")
    bound, lse = torch.zeros_like(out), torch.full((sum(lens_q), hq), -math.inf, dtype=torch.float64, device="cuda")
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        kn, vn = (x.double() for x in kv_of(n))
        g = hq // kn.shape[1]
        kn, vn = kn.repeat_interleave(g, 1), vn.repeat_interleave(g, 1)
        w = torch.einsum("ihd,jhd->hij", q[a:a + lq].double(), kn) * scale
        i = torch.arange(lq, device="cuda")[:, None] + lk - lq
        w = w.masked_fill(torch.arange(lk, device="cuda") > i, -math.inf)
        l = torch.logsumexp(w, -1) if lk else torch.full((hq, lq), -math.inf, dtype=torch.float64, device="cuda")
        p = torch.where(torch.isfinite(l)[..., None], (w - l[..., None]).exp(), 0.0)
        out[a:a + lq] = torch.einsum("hij,jhd->ihd", p, vn)
        bound[a:a + lq] = torch.einsum("hij,jhd->ihd", p, vn.abs())
        lse[a:a + lq] = l.T
        a += lq
    return out, U * (bound + out.abs()) + 1e-30, lse


def check_attn(q, out, lse, ref, scale):
    o, bound, l = ref
    within("out", out, o, bound)
    empty = torch.isinf(l)
    assert (out[empty] == 0).all()
    if lse is not None:
        assert torch.equal(torch.isinf(lse), empty)
        # fp32 scores of up to |l| and a sum of fp32 exponentials
        within("lse", torch.where(empty, 0.0, lse), torch.where(empty, 0.0, l), 2.0 ** -18 * (1.0 + l.abs().nan_to_num(posinf=0)))


PROMPTS = [
    ([1], 1, 1), ([2, 1, 3], 4, 4), ([64], 8, 1), ([127, 128, 129], 8, 2), ([255, 0, 257], 6, 2), ([300, 700, 1024], 8, 4),
    ([1500], 7, 1), ([33, 65], 28, 4), ([5, 40], 128, 1), ([50, 3], 5, 5), ([0, 0, 31, 0], 2, 2), ([2100], 3, 3), ([1000, 1], 40, 2),
]


@pytest.mark.parametrize("lens,hq,hk", PROMPTS, ids=[f"{'-'.join(map(str, a))}x{b}/{c}" for a, b, c in PROMPTS])
@pytest.mark.parametrize("spread", [1.0, 12.0], ids=["flat", "peaked"])
def test_attn_prompts(lens, hq, hk, spread):
    g = gen_of(sum(lens) + hq)
    T, more = sum(lens), 37                                # rows of the buffers past every sequence
    q = rand(g, T + more, hq, D, mul=spread)
    kv = rand(g, T + more, (1 + 2 * hk) * D)               # keys and values as columns of one buffer
    k, v = kv[:, D:(1 + hk) * D].unflatten(1, (hk, D)), kv[:, (1 + hk) * D:].unflatten(1, (hk, D))
    kv[T:] = NAN
    out = torch.full((T + more, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + more, hq), NAN, device="cuda")
    ws = kda.kda_attn_fwd(q, k, v, D ** -0.5, out, lse=lse, cu_seqlens_q=cu_of(lens))
    assert kda.kda_read_device_status(ws) == 0
    assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    ref = ref_attn(q, k, v, D ** -0.5, lens, lens, lambda n: (k[at[n]:at[n + 1]], v[at[n]:at[n + 1]]))
    check_attn(q, out[:T], lse[:T], ref, D ** -0.5)


CACHES = [   # new tokens, keys in the cache (the new ones among them), heads
    ([1], [1], 1, 1), ([1, 1, 1], [1, 77, 400], 8, 2), ([1], [5000], 32, 8), ([1] * 5, [0, 128, 129, 0, 640], 7, 1),
    ([3, 1, 2], [300, 128, 2], 8, 1), ([200, 5], [1000, 700], 4, 4), ([4, 6], [2, 6], 4, 2), ([130], [131], 16, 2),
    ([1, 0, 9], [50, 60, 9], 5, 5), ([1] * 40, list(range(1, 1200, 30)), 28, 4), ([70], [4000], 128, 1),
]


@pytest.mark.parametrize("lens_q,lens_k,hq,hk", CACHES, ids=range(len(CACHES)))
@pytest.mark.parametrize("heads_outside", [False, True], ids=["rows", "heads_first"])
def test_attn_caches(lens_q, lens_k, hq, hk, heads_outside):
    g = gen_of(sum(lens_k) + hq)
    n, room = len(lens_q), max(lens_k) + 19
    q = rand(g, sum(lens_q), hq, D)
    if heads_outside:                                      # a cache laid out [N, Hk, S, 128]
        k, v = (rand(g, n, hk, room, D).transpose(1, 2) for _ in range(2))
    else:
        k, v = (rand(g, n, room, hk, D) for _ in range(2))
    for i, a in enumerate(lens_k):
        k[i, a:] = NAN
        v[i, a:] = NAN
    out = torch.full_like(q, NAN)
    lse = torch.full((sum(lens_q), hq), NAN, device="cuda")
    uniform = len(set(lens_q)) == 1
    for cu in ([cu_of(lens_q), None] if uniform else [cu_of(lens_q)]):
        ws = kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, cu_seqlens_q=cu, seqlens_k=torch.tensor(lens_k, device="cuda"))
        assert kda.kda_read_device_status(ws) == 0
        ref = ref_attn(q, k, v, 0.1, lens_q, lens_k, lambda i: (k[i, :lens_k[i]], v[i, :lens_k[i]]))
        check_attn(q, out, lse, ref, 0.1)


def test_attn_packed_keys_of_other_lengths_and_uniform_batches():
    g = gen_of(5)
    lens_q, lens_k = [3, 100, 1, 40], [50, 300, 200, 7]
    q, k, v = rand(g, sum(lens_q), 8, D), rand(g, sum(lens_k), 2, D), rand(g, sum(lens_k), 2, D)
    out = torch.full_like(q, NAN)
    at = [0] + torch.tensor(lens_k).cumsum(0).tolist()
    kda.kda_attn_fwd(q, k, v, 0.2, out, cu_seqlens_q=cu_of(lens_q), cu_seqlens_k=cu_of(lens_k))
    ref = ref_attn(q, k, v, 0.2, lens_q, lens_k, lambda n: (k[at[n]:at[n + 1]], v[at[n]:at[n + 1]]))
    check_attn(q, out, None, ref, 0.2)
    # without cu_seqlens at all: one sequence
    ref1 = ref_attn(q, k, v, 0.2, [sum(lens_q)], [sum(lens_k)], lambda n: (k, v))
    kda.kda_attn_fwd(q, k, v, 0.2, out)
    check_attn(q, out, None, ref1, 0.2)
    # queries divided evenly over packed keys
    q4 = q[:8].contiguous()
    out4 = torch.full_like(q4, NAN)
    kda.kda_attn_fwd(q4, k, v, 0.2, out4, cu_seqlens_k=cu_of(lens_k))
    ref4 = ref_attn(q4, k, v, 0.2, [2] * 4, lens_k, lambda n: (k[at[n]:at[n + 1]], v[at[n]:at[n + 1]]))
    check_attn(q4, out4, None, ref4, 0.2)


def test_attn_strided_queries_and_outputs():
    g = gen_of(6)
    lens, hq, hk = [200, 90], 6, 3
    T = sum(lens)
    buf = rand(g, hq + 1, T, D + 8)                        # heads outside, rows padded
    q = buf[1:, :, :D].transpose(0, 1)
    k, v = rand(g, T, hk, D), rand(g, T, hk, D)
    obuf = torch.full((T, 2 * hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    out = obuf[:, ::2]
    kda.kda_attn_fwd(q, k, v, 0.1, out, cu_seqlens_q=cu_of(lens))
    ref = ref_attn(q, k, v, 0.1, lens, lens, lambda n: (k[200 * n:200 * n + lens[n]], v[200 * n:200 * n + lens[n]]))
    check_attn(q, out, None, ref, 0.1)
    assert torch.isnan(obuf[:, 1::2]).all()


def test_attn_offsets_past_32_bits():
    """Two sequences at the ends of a cache of over 2^32 elements."""
    n, room, hk = 5, 1 << 20, 8
    k, v = (torch.empty(n, room, hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = gen_of(7)
    lens_k = [0, 0, 0, 0, 1500]
    k[4, :1500], v[4, :1500] = rand(g, 1500, hk, D), rand(g, 1500, hk, D)
    q = rand(g, n, 16, D)
    out, lse = torch.full_like(q, NAN), torch.full((n, 16), NAN, device="cuda")
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, seqlens_k=torch.tensor(lens_k, device="cuda"))
    ref = ref_attn(q, k, v, 0.1, [1] * n, lens_k, lambda i: (k[i, :lens_k[i]], v[i, :lens_k[i]]))
    check_attn(q, out, lse, ref, 0.1)


def test_attn_bad_lengths_write_nothing():
    q, k = torch.zeros(10, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(10, 2, D, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(2, 20, 2, D, dtype=torch.bfloat16, device="cuda")
    i64 = lambda *a: torch.tensor(a, dtype=torch.int64, device="cuda")
    calls = [(k, dict(cu_seqlens_q=i64(0, 5, 4, 10))), (k, dict(cu_seqlens_q=i64(1, 5, 10))), (k, dict(cu_seqlens_q=i64(0, 5, 11))),
             (k, dict(cu_seqlens_q=i64(0, 5, 10), cu_seqlens_k=i64(0, 12, 10))), (cache, dict(cu_seqlens_q=i64(0, 5, 10), seqlens_k=i64(3, 21))),
             (cache, dict(cu_seqlens_q=i64(0, 5, 10), seqlens_k=i64(-1, 3)))]
    for kv, kw in calls:
        out = torch.full_like(q, NAN)
        ws = kda.kda_attn_fwd(q, kv, kv.clone(), 1.0, out, **kw)
        assert kda.kda_read_device_status(ws) == kb.KDA_DEVERR_CU_SEQLENS
        assert torch.isnan(out).all()
        ws2 = kda.kda_attn_fwd(q, k, k.clone(), 1.0, out, workspace=ws)     # the same workspace, a good call
        assert kda.kda_read_device_status(ws2) == 0 and (out == 0).all()


def test_attn_gives_the_same_bits_again_and_on_another_stream():
    g = gen_of(8)
    lens = [700, 1024, 300]
    T = sum(lens)
    q, k, v = rand(g, T, 16, D), rand(g, T, 4, D), rand(g, T, 4, D)
    outs = [torch.full_like(q, NAN) for _ in range(3)]
    kda.kda_attn_fwd(q, k, v, 0.1, outs[0], cu_seqlens_q=cu_of(lens))
    cu = cu_of(lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kda.kda_attn_fwd(q, k, v, 0.1, outs[1], cu_seqlens_q=cu, stream=s)
    with torch.cuda.stream(s):
        kda.kda_attn_fwd(q, k, v, 0.1, outs[2], cu_seqlens_q=cu)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------- linear attention
def ref_lin(q, k, v, ld, scale, lens, init):
    """Token by token over packed [T, H, 128] rows: (out, bound A, state, state of absolute values)."""
    h = q.shape[1]
    decay = ld.double().exp()[:, None, None]
    outs, bounds, finals, finals_abs = [], [], [], []
    a = 0
    for n, L in enumerate(lens):
        s = torch.zeros(h, D, D, dtype=torch.float64, device="cuda") if init is None else init[n].double()
        t = s.abs()
        for i in range(a, a + L):
            qi, ki, vi = q[i].double(), k[i].double(), v[i].double()
            s = decay * s + vi[:, :, None] * ki[:, None, :]
            t = decay * t + vi.abs()[:, :, None] * ki.abs()[:, None, :]
            outs.append(scale * torch.einsum("hvk,hk->hv", s, qi))
            bounds.append(scale * torch.einsum("hvk,hk->hv", t, qi.abs()))
        a += L
        finals.append(s)
        finals_abs.append(t)
    none = torch.zeros(0, h, D, dtype=torch.float64, device="cuda")
    return (torch.stack(outs) if outs else none, torch.stack(bounds) if bounds else none, torch.stack(finals), torch.stack(finals_abs))


def check_state(name, got, ref, absolute):
    bound = 2.0 ** -17 * absolute + 1e-30
    if got.dtype == torch.bfloat16:
        bound = bound + U * 1.01 * ref.abs()
    within(name, got, ref, bound)


def check_lin_out(out, o, A):
    within("out", out, o, U * 1.01 * (o.abs() + A) + 1e-30)
    if o.numel() and o.norm() > 0:
        assert (out.double() - o).norm() / o.norm() <= 2.0 ** -8


LINS = [([1], 1), ([2, 1], 2), ([127], 3), ([128], 2), ([129, 0, 1], 2), ([256, 384], 1), ([300, 700, 1024], 2), ([511], 5), ([33, 64, 65, 100], 4),
        ([0, 0], 2), ([1900], 1)]
DECAYS = {"mixed": lambda h: -(2.0 ** -torch.arange(0.0, h)), "none": lambda h: torch.zeros(h), "strong": lambda h: torch.full((h,), -9.0),
          "forget": lambda h: torch.full((h,), -math.inf), "slow": lambda h: torch.full((h,), -1e-4)}


@pytest.mark.parametrize("lens,h", LINS, ids=[f"{'-'.join(map(str, a))}x{b}" for a, b in LINS])
@pytest.mark.parametrize("decay,states", [("mixed", "f32"), ("none", "none"), ("strong", "bf16"), ("forget", "f32"), ("slow", "mixed")])
def test_lin_fwd(lens, h, decay, states):
    g = gen_of(sum(lens) + h)
    T, more, n = sum(lens), 21, len(lens)
    qkv = rand(g, T + more, 3 * h * D)
    qkv[T:] = NAN
    q, k, v = (x.unflatten(1, (h, D))[None] for x in qkv.split(h * D, 1))
    ld = DECAYS[decay](h).cuda()
    dt = {"f32": (torch.float32,) * 2, "bf16": (torch.bfloat16,) * 2, "none": (None, torch.float32), "mixed": (torch.bfloat16, torch.float32)}[states]
    init = None if dt[0] is None else rand(g, n, h, D, D, dtype=dt[0])
    final = torch.full((n, h, D, D), NAN, dtype=dt[1], device="cuda")
    out = torch.full((1, T + more, h, D), NAN, dtype=torch.bfloat16, device="cuda")
    scale = D ** -0.5
    ws = kda.kda_lin_fwd(q, k, v, ld, scale, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
    assert kda.kda_read_device_status(ws) == 0
    o, A, s, t = ref_lin(q[0], k[0], v[0], ld, scale, lens, init)
    assert torch.isnan(out[0, T:]).all()
    check_lin_out(out[0, :T], o, A)
    check_state("final_state", final, s, t)
    if init is not None and init.dtype == final.dtype:     # the state updated in place, no outputs kept apart
        kda.kda_lin_fwd(q, k, v, ld, scale, out, initial_state=init, final_state=init, cu_seqlens=cu_of(lens))
        assert torch.equal(init, final)


def test_lin_fwd_does_not_let_one_sequence_into_another():
    """A sequence of NaN in the middle of the batch stays where it is."""
    g = gen_of(3)
    lens, h = [200, 61, 300], 2
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    for x in (q, k, v):
        x[0, 200:261] = NAN
    ld = DECAYS["mixed"](h).cuda()
    out = torch.empty_like(q)
    final = torch.empty(3, h, D, D, device="cuda")
    kda.kda_lin_fwd(q, k, v, ld, 0.1, out, final_state=final, cu_seqlens=cu_of(lens))
    for n, (a, b) in ((0, (0, 200)), (2, (261, 561))):
        o, A, s, t = ref_lin(q[0, a:b], k[0, a:b], v[0, a:b], ld, 0.1, [b - a], None)
        check_lin_out(out[0, a:b], o, A)
        check_state("final_state", final[n:n + 1], s, t)


@pytest.mark.parametrize("B,T,h,strided", [(2, 200, 3, False), (3, 1, 2, True), (1, 5, 1, False), (5, 77, 2, True), (2, 0, 2, False)])
def test_lin_fwd_batched(B, T, h, strided):
    g = gen_of(B * T + h)
    if strided:
        q, k, v = (x.unflatten(2, (h, D)) for x in rand(g, B, T, 3 * h * D).split(h * D, 2))
    else:
        q, k, v = (rand(g, B, T, h, D) for _ in range(3))
    ld = DECAYS["mixed"](h).cuda()
    init, final = rand(g, B, h, D, D, dtype=torch.float32), torch.full((B, h, D, D), NAN, device="cuda")
    out = torch.full((B, T, h, D), NAN, dtype=torch.bfloat16, device="cuda")
    kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final)
    flat = [x.reshape(B * T, h, D) for x in (q, k, v, out)]
    o, A, s, t = ref_lin(*flat[:3], ld, 0.1, [T] * B, init)
    check_lin_out(flat[3], o, A)
    check_state("final_state", final, s, t)


def test_lin_fwd_many_units_and_a_long_prompt():
    """More units than the GPU has SMs, and few units with a long prompt: against a 64-bit chunked
    evaluation (the recurrence unrolled over 64 tokens at a time)."""
    for seed, lens, h in ((11, [700, 90, 1300], 96), (12, [9000], 4), (13, [4100, 128, 2500], 8)):
        g = gen_of(seed)
        T = sum(lens)
        q, k, v = (rand(g, 1, T, h, D) for _ in range(3))
        ld = (-(2.0 ** (-8.0 * torch.arange(1, h + 1) / h))).cuda()
        init, final = rand(g, len(lens), h, D, D, dtype=torch.float32), torch.full((len(lens), h, D, D), NAN, device="cuda")
        out = torch.full_like(q, NAN)
        ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu_of(lens))
        assert kda.kda_read_device_status(ws) == 0
        a = 0
        d = ld.double()[:, None]
        for n, L in enumerate(lens):
            s, sa = init[n].double(), init[n].double().abs()
            for c in range(a, a + L, 64):
                m = min(64, a + L - c)
                i = torch.arange(m, device="cuda")
                qc, kc, vc = (x[0, c:c + m].double().transpose(0, 1) for x in (q, k, v))
                gap = (i[:, None] - i).clamp(min=0)
                low = torch.exp(d[..., None] * gap) * (i[:, None] >= i)
                o = (qc @ kc.transpose(1, 2) * low) @ vc + torch.exp(d * (i + 1))[..., None] * (qc @ s.transpose(1, 2))
                A = (qc.abs() @ kc.abs().transpose(1, 2) * low) @ vc.abs() + torch.exp(d * (i + 1))[..., None] * (qc.abs() @ sa.transpose(1, 2))
                check_lin_out(out[0, c:c + m], 0.1 * o.transpose(0, 1), 0.1 * A.transpose(0, 1))
                w = torch.exp(d * (m - 1 - i))[..., None]
                s = torch.exp(d * m)[..., None] * s + (vc * w).transpose(1, 2) @ kc
                sa = torch.exp(d * m)[..., None] * sa + (vc * w).abs().transpose(1, 2) @ kc.abs()
            check_state("final_state", final[n], s, sa)
            a += L


def test_lin_fwd_bad_lengths_write_nothing():
    q = torch.zeros(1, 10, 2, D, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 5, 4, 10], [1, 5, 10], [0, 5, 11]):
        out, final = torch.full_like(q, NAN), torch.full((len(cu) - 1, 2, D, D), NAN, device="cuda")
        ws = kda.kda_lin_fwd(q, q.clone(), q.clone(), torch.zeros(2, device="cuda"), 1.0, out, final_state=final,
                             cu_seqlens=torch.tensor(cu, device="cuda"))
        assert kda.kda_read_device_status(ws) == kb.KDA_DEVERR_CU_SEQLENS
        assert torch.isnan(out).all() and torch.isnan(final).all()


@pytest.mark.parametrize("B,h,states,strided", [(1, 1, "f32", False), (5, 3, "bf16", True), (64, 8, "f32", False), (3, 40, "none", True),
                                                (7, 2, "mixed", False), (0, 4, "f32", False)])
def test_lin_decode(B, h, states, strided):
    g = gen_of(B + h)
    if strided:
        q, k, v = (x.unflatten(1, (h, D)) for x in rand(g, B, 3 * h * D).split(h * D, 1))
    else:
        q, k, v = (rand(g, B, h, D) for _ in range(3))
    ld = DECAYS["mixed"](h).cuda()
    ld[-1] = -math.inf if h > 1 else ld[-1]
    dt = {"f32": (torch.float32,) * 2, "bf16": (torch.bfloat16,) * 2, "none": (None, torch.float32), "mixed": (torch.float32, torch.bfloat16)}[states]
    init = None if dt[0] is None else rand(g, B, h, D, D, dtype=dt[0])
    final = torch.full((B, h, D, D), NAN, dtype=dt[1], device="cuda")
    out = torch.full((B, h, D), NAN, dtype=torch.bfloat16, device="cuda")
    kda.kda_lin_decode(q, k, v, ld, 0.3, out, initial_state=init, final_state=final)
    s0 = 0.0 if init is None else init.double()
    dec = ld.double().exp()[:, None, None]
    vk = v.double()[..., None] * k.double()[..., None, :]
    s, t = dec * s0 + vk, dec * (s0 if init is None else s0.abs()) + vk.abs()
    o = 0.3 * (s @ q.double()[..., None]).squeeze(-1)
    A = 0.3 * (t @ q.double().abs()[..., None]).squeeze(-1)
    within("out", out, o, U * 1.01 * o.abs() + 2.0 ** -16 * A + 1e-30)
    check_state("final_state", final, s, t)
    if init is not None and dt[0] == dt[1]:
        kda.kda_lin_decode(q, k, v, ld, 0.3, out, initial_state=init, final_state=init)
        assert torch.equal(init, final)


def test_prompt_then_steps_is_one_longer_prompt():
    """kda_lin_fwd over 140 tokens, then 5 steps on its state, against kda_lin_fwd over all 145."""
    g = gen_of(21)
    T, S, h = 140, 5, 3
    q, k, v = (rand(g, 1, T + S, h, D) for _ in range(3))
    ld = DECAYS["mixed"](h).cuda()
    state = torch.empty(1, h, D, D, device="cuda")
    out = torch.empty_like(q)
    kda.kda_lin_fwd(q[:, :T], k[:, :T], v[:, :T], ld, 0.1, out[:, :T], final_state=state)
    for i in range(T, T + S):
        kda.kda_lin_decode(q[:, i], k[:, i], v[:, i], ld, 0.1, out[:, i], initial_state=state, final_state=state)
    o, A, s, t = ref_lin(q[0], k[0], v[0], ld, 0.1, [T + S], None)
    check_lin_out(out[0], o, A)
    check_state("state", state, s, t)
