"""The token mixers that stand beside Kimi Delta Attention in a hybrid stack, as measured cases.

Four operators of one layer family (head dim 128, bf16 tokens, packed sequences):

  norm_rope   RMS norm of every query and key head and the rotary position rotation, one pass
  attn        causal softmax attention with grouped heads over packed prompts, prompts that
              continue a cache, and single tokens over a cache
  lin_fwd     linear attention with a decay for each head over packed prompts (chunked)
  lin_step    the same recurrence for one token of every sequence

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes
what a program holds before the call, ``run`` is one call, ``work`` what it cannot do without,
``exact`` the definition in 64 bits.  With ``own`` false ``run`` computes the plain form in
elementary torch operations in 32 bits; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

D = 128
EPS = 1e-6
# (query heads, key/value heads): equal, grouped by 2 to 8, one shared head, an odd group
HEADS = [(32, 8), (64, 8), (32, 32), (16, 2), (28, 4), (8, 1), (5, 5), (40, 8)]
LIN_HEADS = [4, 5, 8, 16, 32, 40, 64, 96]
MAX_SCORES = 64 * 8192 * 8192      # padded scores of the largest listed prompt
MAX_LIN = 45661 * 64               # token-heads of the largest listed linear prompt


def listed():
    return [
        # one decode step of eight requests: a latency
        {"name": "rope step", "op": "norm_rope", "tokens": 8, "hq": 32, "hk": 8, "rot": 128, "interleaved": False, "fused": True},
        # the three prompts of the packed3 workload, half of each head rotated, adjacent pairs
        {"name": "rope packed", "op": "norm_rope", "tokens": 2024, "hq": 32, "hk": 8, "rot": 64, "interleaved": True, "fused": True},
        # a long prompt
        {"name": "rope long", "op": "norm_rope", "tokens": 32768, "hq": 64, "hk": 8, "rot": 128, "interleaved": False, "fused": True},
        # the packed3 prompts: ragged, few tiles
        {"name": "attn packed", "op": "attn", "kind": "prompt", "lens_q": "300,700,1024", "lens_k": "300,700,1024", "hq": 32, "hk": 8, "fused": True, "lse": True},
        # one long prompt: bound by the tensor cores
        {"name": "attn long", "op": "attn", "kind": "prompt", "lens_q": "8192", "lens_k": "8192", "hq": 64, "hk": 8, "fused": False, "lse": False},
        # one request decoding over a long cache: one row of work for the whole GPU
        {"name": "attn step one", "op": "attn", "kind": "step", "lens_q": "1", "lens_k": "32767", "hq": 32, "hk": 8, "fused": False, "lse": False},
        # a decode batch over caches of different lengths
        {"name": "attn step batch", "op": "attn", "kind": "step", "lens_q": ",".join(["1"] * 32),
         "lens_k": ",".join(str(67 + 262 * i) for i in range(32)), "hq": 32, "hk": 8, "fused": False, "lse": False},
        # the packed3 workload's lengths and heads: three units' worth of chunks for each SM
        {"name": "lin packed", "op": "lin_fwd", "lens": "300,700,1024", "h": 96, "init": "f32", "final": "f32"},
        # the long workload: 32 chains of 32,768 tokens
        {"name": "lin long", "op": "lin_fwd", "lens": "32768", "h": 32, "init": "none", "final": "bf16"},
        # eight prompts of mixed lengths, 45,661 tokens
        {"name": "lin mix", "op": "lin_fwd", "lens": "8000,7777,6401,5003,1200,63,8129,9088", "h": 64, "init": "f32", "final": "f32"},
        # one request: a latency
        {"name": "lin step one", "op": "lin_step", "batch": 1, "h": 32, "init": "f32", "final": "f32"},
        # a decode batch: bound by the states' traffic
        {"name": "lin step batch", "op": "lin_step", "batch": 64, "h": 64, "init": "f32", "final": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(n):
    """A drawn size is ragged: the multiples of 1024 are among the listed ones."""
    return n + 1 if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(["norm_rope", "attn", "attn", "lin_fwd", "lin_fwd", "lin_step"])
    if op == "norm_rope":
        hq, hk = rng.choice(HEADS)
        return {"op": op, "tokens": _odd(_log(rng, 1, 32768 * 72 // (hq + hk) if hq + hk > 72 else 32768)), "hq": hq, "hk": hk,
                "rot": rng.choice([32, 64, 128]), "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5}
    if op == "attn":
        hq, hk = rng.choice(HEADS)
        kind = rng.choice(["prompt", "continue", "step"])
        if kind == "prompt":
            n = _log(rng, 1, 8)
            lens_q = [_odd(_log(rng, 1, 8192)) for _ in range(n)]
            lens_k = lens_q
        elif kind == "continue":
            n = _log(rng, 1, 4)
            lens_q = [_odd(_log(rng, 1, 1024)) for _ in range(n)]
            lens_k = [_odd(a + _log(rng, 1, 16384)) for a in lens_q]
        else:
            n = _log(rng, 1, 64)
            lens_q = [1] * n
            lens_k = [_odd(_log(rng, 1, 32768)) for _ in range(n)]
        while n > 1 and (n * hq * max(lens_q) * max(lens_k) > MAX_SCORES or n * max(lens_k) * hk > 32 * 32768 * 8):
            n -= 1
            lens_q, lens_k = lens_q[:n], lens_k[:n]
        return {"op": op, "kind": kind, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)), "hq": hq, "hk": hk,
                "fused": kind == "prompt" and rng.random() < 0.5, "lse": rng.random() < 0.5}
    if op == "lin_fwd":
        h = rng.choice(LIN_HEADS)
        lens = [_odd(_log(rng, 1, 32768)) for _ in range(_log(rng, 1, 8))]
        while len(lens) > 1 and len(lens) * max(lens) * h > MAX_LIN:
            lens.remove(max(lens))
        lens = [_odd(min(a, MAX_LIN // h)) for a in lens]
        return {"op": op, "lens": ",".join(map(str, lens)), "h": h, "init": rng.choice(["none", "f32", "bf16"]), "final": rng.choice(["f32", "bf16"])}
    h = rng.choice(LIN_HEADS)
    return {"op": op, "batch": _log(rng, 1, 4096 // h), "h": h, "init": rng.choice(["none", "f32", "bf16"]), "final": rng.choice(["f32", "bf16"])}


def _ints(text):
    return [int(a) for a in text.split(",")]


def _cu(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(dev)


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16, mul=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * mul).to(dtype)

    op = case["op"]
    s = {"op": op}
    if op == "norm_rope":
        t, hq, hk, rot = case["tokens"], case["hq"], case["hk"], case["rot"]
        if case["fused"]:      # q and k as the projection leaves them: columns of one qkv buffer
            qkv = rand(t, (hq + 2 * hk) * D, mul=2.0)
            s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
            s["k"] = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
        else:
            s["q"], s["k"] = rand(t, hq, D, mul=2.0), rand(t, hk, D, mul=2.0)
        s["q_weight"] = rand(D, dtype=torch.float32, mul=0.2) + 1.0
        s["k_weight"] = rand(D, dtype=torch.float32, mul=0.2) + 1.0
        reach = 40960
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(reach, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # several requests' positions, each counting up from a start of its own
        at = torch.arange(t, device=dev)
        start = torch.randint(0, reach - 32768, (64,), generator=gen, device=dev)
        s["positions"] = start[at % 64 if t <= 64 else at * 64 // t] + (at if t > 64 else 0)
        s["interleaved"] = case["interleaved"]
        s["q_out"] = torch.empty(t, hq, D, device=dev, dtype=torch.bfloat16)
        s["k_out"] = torch.empty(t, hk, D, device=dev, dtype=torch.bfloat16)
    elif op == "attn":
        lens_q, lens_k, hq, hk = _ints(case["lens_q"]), _ints(case["lens_k"]), case["hq"], case["hk"]
        tq, n = sum(lens_q), len(lens_q)
        s["cu_q"] = _cu(lens_q, dev)
        s["max_q"], s["max_k"] = max(lens_q), max(lens_k)
        s["q"] = rand(tq, hq, D, mul=1.5)
        if case["kind"] == "prompt":
            s["k"] = rand(tq, hk, D)
            if case["fused"]:  # v where the projection left it
                s["v"] = rand(tq, (hq + 2 * hk) * D)[:, (hq + hk) * D:].unflatten(1, (hk, D))
            else:
                s["v"] = rand(tq, hk, D)
            s["lens_k"] = None
        else:                  # a cache of fixed room for each sequence
            room = (max(lens_k) + 79) // 80 * 80
            s["k"], s["v"] = rand(n, room, hk, D), rand(n, room, hk, D)
            s["lens_k"] = torch.tensor(lens_k, dtype=torch.int64, device=dev)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(tq, hq, D, device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.empty(tq, hq, device=dev) if case["lse"] else None
    else:
        h = case["h"]
        if op == "lin_fwd":
            lens = _ints(case["lens"])
            n, shape = len(lens), (1, sum(lens), h, D)
            s["cu"], s["max_len"] = _cu(lens, dev), max(lens)
        else:
            n = case["batch"]
            shape = (n, h, D)
        s["q"], s["k"], s["v"] = rand(*shape), rand(*shape), rand(*shape)
        # decays that forget within a few tokens up to some hundreds
        s["log_decay"] = -(2.0 ** (-8.0 * torch.arange(1, h + 1, device=dev, dtype=torch.float32) / h)) * (
            1.0 + 0.1 * torch.rand(h, generator=gen, device=dev))
        s["scale"] = D ** -0.5
        s["init"] = None if case["init"] == "none" else rand(n, h, D, D, dtype=DT[case["init"]])
        s["final"] = torch.empty(n, h, D, D, device=dev, dtype=DT[case["final"]])
        s["out"] = torch.empty(shape, device=dev, dtype=torch.bfloat16)
    return s


# ------------------------------ one pass -------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_norm_rope(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], s["q_out"], s["k_out"],
                         eps=EPS, flags=kda.KDA_FLAG_ROPE_INTERLEAVED if s["interleaved"] else 0)
    return s["q_out"], s["k_out"]


def _own_attn(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_attn_fwd(s["q"], s["k"], s["v"], s["scale"], s["out"], lse=s["lse"], cu_seqlens_q=s["cu_q"], seqlens_k=s["lens_k"])
    return (s["out"],) if s["lse"] is None else (s["out"], s["lse"])


def _own_lin_fwd(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_lin_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["out"], initial_state=s["init"], final_state=s["final"],
                    cu_seqlens=s["cu"])
    return s["out"], s["final"]


def _own_lin_step(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_lin_decode(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["out"], initial_state=s["init"], final_state=s["final"])
    return s["out"], s["final"]


_own = {"norm_rope": _own_norm_rope, "attn": _own_attn, "lin_fwd": _own_lin_fwd, "lin_step": _own_lin_step}


def _norm_rope_one(x, weight, cos, sin, interleaved):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., 2 * half:]], -1).to(torch.bfloat16)


def _plain_norm_rope(s):
    cos, sin = s["cos_sin"][s["positions"]][:, None].chunk(2, -1)
    return (_norm_rope_one(s["q"], s["q_weight"], cos, sin, s["interleaved"]),
            _norm_rope_one(s["k"], s["k_weight"], cos, sin, s["interleaved"]))


def _padded(x, cu, most):
    """[T, ...] packed rows as float [N, most, ...], zero past each sequence's end, and which rows are real."""
    at = torch.arange(most, device=x.device)
    real = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=x.shape[0] - 1)
    y = x[rows].float()
    return y.masked_fill_(~real.reshape(real.shape + (1,) * (x.dim() - 1)), 0.0), real


def _packed(y, cu, total):
    """Rows of [N, most, ...] back in packed order."""
    t = torch.arange(total, device=y.device)
    n = torch.searchsorted(cu[1:], t, right=True)
    return y[n, t - cu[n]]


def _plain_attn(s):
    q, cu = s["q"], s["cu_q"]
    qp, _ = _padded(q, cu, s["max_q"])
    len_q = cu[1:] - cu[:-1]
    if s["lens_k"] is None:
        kp, vp = _padded(s["k"], cu, s["max_k"])[0], _padded(s["v"], cu, s["max_k"])[0]
        len_k = len_q
    else:
        kp, vp = s["k"][:, :s["max_k"]].float(), s["v"][:, :s["max_k"]].float()
        len_k = s["lens_k"]
        vp.masked_fill_((torch.arange(s["max_k"], device=q.device) >= len_k[:, None])[..., None, None], 0.0)
    n, lq, hq, _ = qp.shape
    lk, hk = kp.shape[1], kp.shape[2]
    qp = qp.reshape(n, lq, hk, hq // hk, D).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, D)      # group's rows side by side
    w = torch.matmul(qp * s["scale"], kp.permute(0, 2, 3, 1)).reshape(n, hk, hq // hk, lq, lk)
    i = torch.arange(lq, device=q.device)[:, None] + (len_k - len_q)[:, None, None]
    seen = torch.arange(lk, device=q.device) <= i.clamp(max=(len_k - 1)[:, None, None])
    w.masked_fill_(~seen[:, None, None], float("-inf"))
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(n, hk, -1, lk), vp.permute(0, 2, 1, 3)).reshape(n, hk, hq // hk, lq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, D)
    out = _packed(o, cu, q.shape[0]).to(torch.bfloat16)
    if s["lse"] is None:
        return (out,)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(n, lq, hq)
    return out, _packed(lse, cu, q.shape[0])


def _plain_lin_fwd(s):
    """Chunks of 128 tokens, every chunk at once: the products inside a chunk, each chunk's own
    sum of v k^T, and the sums carried from chunk to chunk as one product with the decays between them."""
    C = 128
    q, cu, ld = s["q"][0], s["cu"], s["log_decay"]
    lens = cu[1:] - cu[:-1]
    nc = (s["max_len"] + C - 1) // C
    n, h = lens.shape[0], q.shape[1]
    pad = nc * C - lens                                      # sequences end where their last chunk ends
    at = torch.arange(nc * C, device=q.device)
    real = at >= pad[:, None]
    rows = (cu[:-1, None] + at - pad[:, None]).clamp(min=0)

    def chunks(x):
        y = x[0][rows].float().masked_fill_(~real[..., None, None], 0.0)
        return y.reshape(n, nc, C, h, D).permute(0, 3, 1, 2, 4)

    qc, kc, vc = chunks(s["q"]) * s["scale"], chunks(s["k"]), chunks(s["v"])
    i = torch.arange(C, device=q.device)
    gap = i[:, None] - i
    inner = torch.exp(ld[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
    o = torch.matmul(torch.matmul(qc, kc.transpose(-1, -2)) * inner[:, None], vc)
    to_end = torch.exp(ld[:, None] * (C - 1 - i))
    sums = torch.matmul((vc * to_end[:, None, :, None]).transpose(-1, -2), kc)               # [n, h, nc, V, K]
    c = torch.arange(nc + 1, device=q.device)
    hop = c[:, None] - 1 - c[:nc]
    carry = torch.exp(ld[:, None, None] * C * hop.clamp(min=0)) * (hop >= 0)
    before = torch.matmul(carry, sums.flatten(3)).unflatten(-1, (D, D))                      # [n, h, nc + 1, V, K]
    since = torch.exp(ld[:, None] * (i + 1))
    o = o + torch.matmul(qc * since[:, None, :, None], before[:, :, :nc].transpose(-1, -2))
    final = before[:, :, nc]
    if s["init"] is not None:
        init = s["init"].float()
        age = torch.exp(ld[:, None] * (at - pad[:, None] + 1).clamp(min=0)[:, None]).reshape(n, h, nc, C, 1)
        o = o + torch.matmul(qc * age, init[:, :, None].transpose(-1, -2))
        final = final + torch.exp(ld * lens[:, None])[..., None, None] * init
    o = o.permute(0, 2, 3, 1, 4).reshape(n, nc * C, h, D)
    t = torch.arange(q.shape[0], device=q.device)
    m = torch.searchsorted(cu[1:], t, right=True)
    out = o[m, t - cu[m] + pad[m]].to(torch.bfloat16)[None]
    return out, final.to(s["final"].dtype)


def _plain_lin_step(s):
    state = s["v"].float()[..., :, None] * s["k"].float()[..., None, :]
    if s["init"] is not None:
        state = state + torch.exp(s["log_decay"])[:, None, None] * s["init"].float()
    out = torch.matmul(state, s["q"].float()[..., None]).squeeze(-1) * s["scale"]
    return out.to(torch.bfloat16), state.to(s["final"].dtype)


_plain = {"norm_rope": _plain_norm_rope, "attn": _plain_attn, "lin_fwd": _plain_lin_fwd, "lin_step": _plain_lin_step}


# ------------------------------ what a pass cannot do without ----------------------------------
SIZE = {"none": 0, "f32": 4, "bf16": 2}


def work(case):
    op = case["op"]
    if op == "norm_rope":
        t, heads = case["tokens"], case["hq"] + case["hk"]
        return {"bytes": t * (2 * heads * D * 2 + 8 + case["rot"] * 4), "flops": t * heads * (4 * D + 3 * case["rot"])}
    if op == "attn":
        lens_q, lens_k, hq, hk = _ints(case["lens_q"]), _ints(case["lens_k"]), case["hq"], case["hk"]
        # query i of a sequence sees keys 0 .. i + lk - lq
        pairs = sum(lq * (lk - lq) + lq * (lq + 1) // 2 for lq, lk in zip(lens_q, lens_k))
        return {"bytes": sum(lens_q) * hq * (2 * D * 2 + (4 if case["lse"] else 0)) + sum(lens_k) * hk * 2 * D * 2, "flops": 4 * D * hq * pairs}
    h = case["h"]
    if op == "lin_fwd":
        lens = _ints(case["lens"])
        tokens, units = sum(lens) * h, len(lens) * h
        # chunked in 128 tokens: the two triangular products, the state's update and its read-out
        return {"bytes": tokens * 4 * D * 2 + units * D * D * (SIZE[case["init"]] + SIZE[case["final"]]), "flops": tokens * (2 * 128 * D + 4 * D * D)}
    units = case["batch"] * h
    return {"bytes": units * (4 * D * 2 + D * D * (SIZE[case["init"]] + SIZE[case["final"]])), "flops": units * 5 * D * D}


# ------------------------------ the definition in 64 bits ---------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return _exact_norm_rope(s, "q"), _exact_norm_rope(s, "k")
    if op == "attn":
        return _exact_attn(s, _ints(case["lens_q"]), _ints(case["lens_k"]))
    if op == "lin_step":
        return _exact_lin(s["q"][:, None], s["k"][:, None], s["v"][:, None], s, [1] * case["batch"], lambda o: o[:, 0])
    lens = _ints(case["lens"])
    if max(lens) * len(lens) * case["h"] > 16 * MAX_LIN:
        return None
    cut = [torch.nn.utils.rnn.pad_sequence(s[x][0].split(lens), batch_first=True) for x in "qkv"]
    return _exact_lin(*cut, s, lens, lambda o: torch.cat([o[a, :b] for a, b in enumerate(lens)])[None])


def _exact_norm_rope(s, which):
    x, weight = s[which].double(), s[which + "_weight"].double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight
    half = s["cos_sin"].shape[1] // 2
    # each pair as a complex number, turned by its angle
    turn = torch.complex(*s["cos_sin"].double()[s["positions"]].split(half, 1))[:, None]
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attn(s, lens_q, lens_k):
    q, hq = s["q"], s["q"].shape[1]
    hk = s["k"].shape[-2]
    out = torch.zeros(q.shape, device=q.device, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], device=q.device, dtype=torch.float64)
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        k, v = (s[x][a:a + lq] if s["lens_k"] is None else s[x][n, :lk] for x in "kv")
        for h in range(hk):
            kh, vh = k[:, h].double(), v[:, h].double()
            g = slice(h * hq // hk, (h + 1) * hq // hk)
            for i in range(0, lq, 512):
                j = min(lq, i + 512)
                reach = j + lk - lq                           # keys that the block's last row sees
                w = torch.einsum("tgd,kd->gtk", q[a + i:a + j, g].double(), kh[:reach]) * s["scale"]
                last = torch.arange(i, j, device=q.device) + lk - lq
                w = w.masked_fill(torch.arange(reach, device=q.device) > last[:, None], float("-inf"))
                l = torch.logsumexp(w, -1)
                out[a + i:a + j, g] = torch.einsum("gtk,kd->tgd", (w - l[..., None]).exp(), vh[:reach])
                lse[a + i:a + j, g] = l.T
        a += lq
    return (out,) if s["lse"] is None else (out, lse)


def _exact_lin(q, k, v, s, lens, back):
    """Token by token: S <- exp(log_decay) S + v k^T, out = scale S q.  A sequence that has ended keeps its state."""
    n, t, h, _ = q.shape
    state = torch.zeros(n, h, D, D, device=q.device, dtype=torch.float64) if s["init"] is None else s["init"].double()
    decay = s["log_decay"].double().exp()
    length = torch.tensor(lens, device=q.device)
    alive = torch.arange(t, device=q.device)[:, None] < length                                # [t, n]
    factor = torch.where(alive[..., None], decay, 1.0)[..., None, None]
    out = torch.empty(n, t, h, D, device=q.device, dtype=torch.float64)
    v = v.double() * alive.T[..., None, None]
    for i in range(t):
        state.mul_(factor[i]).addcmul_(v[:, i, :, :, None], k[:, i, :, None, :].double())
        out[:, i] = torch.matmul(state, q[:, i, :, :, None].double()).squeeze(-1)
    return back(out * s["scale"]), state
