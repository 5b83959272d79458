"""What a hybrid layer needs around its token mixers when it serves, as measured cases.

Four operators of one layer (head dim 128, bf16 tokens, packed sequences):

  residual  the norm after a block, its gate and residual scale, the sum with the residual stream and
            the norm before the next block, one pass
  gated     RMS norm of every head of a mixer's output times its activated gate
  append    new keys and values into a cache held in 4 bits
  attn      causal softmax attention with grouped heads over that cache: single tokens, a few
            drafted tokens, prompts that continue

A cache row (of a sequence, position and key head) has 144 bytes: 64 of the key's codes (byte i holds
channel 2 i in its low half and 2 i + 1 in its high half), 64 of the value's, and eight bf16 numbers: the
key's scale and zero for channels 0..63, those for 64..127, then the value's four.  A channel
stands for scale * code + zero, with zero the smallest value of its 64, scale a 15th of their
range rounded to bf16, and the code rounded to the nearest, ties to even.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes
what a program holds before the call, ``run`` is one call, ``work`` what it cannot do without,
``exact`` the definition in 64 bits.  With ``own`` false ``run`` computes the plain form in
elementary torch operations; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

D = 128
EPS = 1e-6
ROW = 144                          # bytes of a cache row
# (query heads, key/value heads): grouped by 4 and 8, equal, one shared head, odd groups
HEADS = [(32, 8), (64, 8), (32, 32), (16, 2), (28, 4), (8, 1), (5, 5), (40, 8)]
GATED_HEADS = [4, 5, 8, 16, 32, 40, 64, 96]
MAX_SCORES = 3 * 64 * 1024 * 17408  # padded scores of the largest listed call
MAX_ROWS = 16 * 32767 * 8           # padded cache rows of the largest listed call
MAX_NORM = 32768 * 4096             # elements of the largest listed residual stream
MAX_TOKENS = 45661                  # of the largest listed prompts


def listed():
    return [
        # one decode step of eight requests: a latency
        {"name": "residual step", "op": "residual", "tokens": 8, "dim": 4096, "res": "bf16", "post": False, "gate": "none"},
        # three prompts of 2,024 tokens, a width that is no power of two, the stream in fp32, a gated block between two norms
        {"name": "residual packed", "op": "residual", "tokens": 2024, "dim": 2304, "res": "f32", "post": True, "gate": "token"},
        # a long prompt: bound by memory
        {"name": "residual long", "op": "residual", "tokens": 32768, "dim": 4096, "res": "bf16", "post": True, "gate": "none"},
        # one decode step of eight requests
        {"name": "gated step", "op": "gated", "tokens": 8, "h": 32, "silu": False, "fused": True},
        # eight prompts of mixed lengths, 45,661 tokens; the gate where its projection left it
        {"name": "gated mix", "op": "gated", "tokens": 45661, "h": 64, "silu": True, "fused": True},
        # one token of 32 requests into their caches
        {"name": "append step", "op": "append", "lens_q": ",".join(["1"] * 32), "lens_k": ",".join(str(67 + 262 * i) for i in range(32)),
         "hk": 8, "order": "heads", "fused": True, "values": False},
        # the eight prompts of 45,661 tokens, which go on with the values that the cache stands for
        {"name": "append mix", "op": "append", "lens_q": "8000,7777,6401,5003,1200,63,8129,9088",
         "lens_k": "8000,7777,6401,5003,1200,63,8129,9088", "hk": 8, "order": "heads", "fused": True, "values": True},
        # one request decoding over a long cache: one row of work for the whole GPU
        {"name": "kv4 step one", "op": "attn", "kind": "step", "lens_q": "1", "lens_k": "32767", "hq": 32, "hk": 8, "order": "heads", "lse": False},
        # a decode batch over caches of different lengths
        {"name": "kv4 step batch", "op": "attn", "kind": "step", "lens_q": ",".join(["1"] * 32),
         "lens_k": ",".join(str(67 + 262 * i) for i in range(32)), "hq": 32, "hk": 8, "order": "heads", "lse": False},
        # a decode batch over long caches: bound by their traffic
        {"name": "kv4 step long", "op": "attn", "kind": "step", "lens_q": ",".join(["1"] * 16),
         "lens_k": ",".join(str(5002 + 1851 * i) for i in range(16)), "hq": 64, "hk": 8, "order": "rows", "lse": False},
        # four drafted tokens of each request, checked together
        {"name": "kv4 drafts", "op": "attn", "kind": "draft", "lens_q": ",".join(["4"] * 24),
         "lens_k": ",".join(str(71 + 349 * i) for i in range(24)), "hq": 32, "hk": 8, "order": "heads", "lse": False},
        # prompts that continue: bound by the tensor cores
        {"name": "kv4 continue", "op": "attn", "kind": "continue", "lens_q": "1024,517,33", "lens_k": "17408,9001,16000", "hq": 64, "hk": 8,
         "order": "heads", "lse": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(n):
    """A drawn size is ragged: the multiples of 1024 are among the listed ones."""
    return n + 1 if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(["residual", "gated", "append", "attn", "attn", "attn"])
    if op == "residual":
        dim = rng.choice([256, 1000, 2048, 2304, 4096, 5120, 8192]) if rng.random() < 0.5 else 8 * _log(rng, 1, 1024)
        return {"op": op, "tokens": _odd(_log(rng, 1, min(32768, MAX_NORM // dim))), "dim": dim, "res": rng.choice(["bf16", "f32"]),
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "token", "channel"])}
    if op == "gated":
        h = rng.choice(GATED_HEADS)
        return {"op": op, "tokens": _odd(_log(rng, 1, MAX_TOKENS * 64 // max(h, 64))), "h": h, "silu": rng.random() < 0.5, "fused": rng.random() < 0.5}
    order = rng.choice(["heads", "rows"])
    if op == "append":
        hk = rng.choice([1, 2, 4, 5, 8])
        n = _log(rng, 1, 64)
        lens_q = [1] * n if rng.random() < 0.4 else [_odd(_log(rng, 1, 8192)) for _ in range(n)]
        lens_k = [a + (0 if rng.random() < 0.5 else _log(rng, 1, 16384)) for a in lens_q]
        while n > 1 and (sum(lens_q) > MAX_TOKENS or n * max(lens_k) * hk > MAX_ROWS // 4):
            n -= 1
            lens_q, lens_k = lens_q[:n], lens_k[:n]
        return {"op": op, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)), "hk": hk, "order": order,
                "fused": rng.random() < 0.5, "values": rng.random() < 0.5}
    hq, hk = rng.choice(HEADS)
    kind = rng.choice(["step", "step", "draft", "continue"])
    if kind == "step":
        n = _log(rng, 1, 64)
        lens_q = [1] * n
        lens_k = [_odd(_log(rng, 1, 32768)) for _ in range(n)]
    elif kind == "draft":
        n = _log(rng, 1, 32)
        lens_q = [rng.randint(1, 8) for _ in range(n)]
        lens_k = [_odd(a + _log(rng, 1, 16384)) for a in lens_q]
    else:
        n = _log(rng, 1, 4)
        lens_q = [_odd(_log(rng, 1, 1024)) for _ in range(n)]
        lens_k = [_odd(a + _log(rng, 1, 16384)) for a in lens_q]
    while n > 1 and (n * hq * max(lens_q) * max(lens_k) > MAX_SCORES or n * max(lens_k) * hk > MAX_ROWS):
        n -= 1
        lens_q, lens_k = lens_q[:n], lens_k[:n]
    return {"op": op, "kind": kind, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)), "hq": hq, "hk": hk,
            "order": order, "lse": rng.random() < 0.5}


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
    if op == "residual":
        t, d = case["tokens"], case["dim"]
        s["y"] = rand(t, d, mul=3.0)
        s["residual"] = rand(t, d, dtype=DT[case["res"]], mul=2.0)
        s["pre_weight"] = rand(d, dtype=torch.float32, mul=0.2) + 1.0
        s["post_weight"] = rand(d, dtype=torch.float32, mul=0.2) + 1.0 if case["post"] else None
        # one gate for every token and channel, or one for every channel
        s["gate"] = None if case["gate"] == "none" else rand(t, d) if case["gate"] == "token" else rand(1, d).expand(t, d)
        s["scale"] = 0.25
        s["residual_out"], s["out"] = torch.empty_like(s["residual"]), torch.empty_like(s["y"])
    elif op == "gated":
        t, h = case["tokens"], case["h"]
        s["x"] = rand(t, h, D)
        # the gate among a projection's other columns, or by itself
        s["gate"] = rand(t, 2 * h * D)[:, h * D:].unflatten(1, (h, D)) if case["fused"] else rand(t, h, D)
        s["weight"] = rand(D, dtype=torch.float32, mul=0.2) + 1.0
        s["silu"] = case["silu"]
        s["out"] = torch.empty_like(s["x"])
    else:
        lens_q, lens_k, hk = _ints(case["lens_q"]), _ints(case["lens_k"]), case["hk"]
        tq, n = sum(lens_q), len(lens_q)
        room = (max(lens_k) + 79) // 80 * 80
        s["cu_q"] = None if max(lens_q) == 1 else _cu(lens_q, dev)
        s["lens_k"] = torch.tensor(lens_k, dtype=torch.int64, device=dev)
        s["max_q"], s["max_k"] = max(lens_q), max(lens_k)
        if case["order"] == "heads":
            s["cache"] = torch.zeros(n, hk, room, ROW, dtype=torch.uint8, device=dev).transpose(1, 2)
        else:
            s["cache"] = torch.zeros(n, room, hk, ROW, dtype=torch.uint8, device=dev)
        if op == "append":
            if case["fused"]:      # as the projection leaves them, the queries' columns in front
                qkv = rand(tq, 4 * hk * D)
                s["k"], s["v"] = (x.unflatten(1, (hk, D)) for x in qkv[:, 2 * hk * D:].split(hk * D, 1))
            else:
                s["k"], s["v"] = rand(tq, hk, D), rand(tq, hk, D)
            values = case["values"]
            s["k_out"], s["v_out"] = (torch.empty(tq, hk, D, device=dev, dtype=torch.bfloat16) if values else None for _ in "kv")
        else:
            hq = case["hq"]
            # keys whose channels lie around means of their own, values around zero; rows up to the room are filled,
            # as those of an earlier, longer request would be
            mean = rand(hk, D, dtype=torch.float32, mul=0.5)
            for i in range(n):
                k = (torch.randn(room, hk, D, generator=gen, device=dev) + mean).to(torch.bfloat16)
                s["cache"][i] = _rows(k, rand(room, hk, D))
            s["q"] = rand(tq, hq, D, mul=1.5)
            s["scale"] = D ** -0.5
            s["out"] = torch.empty(tq, hq, D, device=dev, dtype=torch.bfloat16)
            s["lse"] = torch.empty(tq, hq, device=dev) if case["lse"] else None
    return s


# ------------------------------ one pass -------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_residual(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_residual_norm(s["y"], s["residual"], s["pre_weight"], s["out"], residual_out=s["residual_out"], post_weight=s["post_weight"],
                          gate=s["gate"], scale=s["scale"], eps=EPS)
    return s["residual_out"], s["out"]


def _own_gated(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_gated_norm(s["x"], s["gate"], s["weight"], s["out"], eps=EPS, flags=kda.KDA_FLAG_GATE_SILU if s["silu"] else 0)
    return s["out"]


def _own_append(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_qcache_append(s["k"], s["v"], s["cache"], s["lens_k"], cu_seqlens=s["cu_q"], k_out=s["k_out"], v_out=s["v_out"])
    return (s["cache"],) if s["k_out"] is None else (s["cache"], s["k_out"], s["v_out"])


def _own_attn(s):
    import gated_delta_rule_36_gb300 as kda
    kda.kda_attn_qcache_fwd(s["q"], s["cache"], s["scale"], s["out"], s["lens_k"], lse=s["lse"], cu_seqlens_q=s["cu_q"])
    return (s["out"],) if s["lse"] is None else (s["out"], s["lse"])


_own = {"residual": _own_residual, "gated": _own_gated, "append": _own_append, "attn": _own_attn}


def _norm(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _plain_residual(s):
    u = s["y"].float()
    if s["post_weight"] is not None:
        u = _norm(u, s["post_weight"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + s["scale"] * u
    return r.to(s["residual"].dtype), _norm(r, s["pre_weight"]).to(torch.bfloat16)


def _plain_gated(s):
    g = s["gate"].float()
    a = 1.0 / (1.0 + torch.exp(-g))
    return (_norm(s["x"].float(), s["weight"]) * (g * a if s["silu"] else a)).to(torch.bfloat16)


def _codes(x):
    """Codes [.., 128], scales and zeros [.., 2] of bf16 vectors; in 64 bits, since a difference next to the border
    between two codes has to fall on its own side."""
    g = x.double().unflatten(-1, (2, D // 2))
    low = g.amin(-1)
    scale = ((g.amax(-1) - low) / 15).to(torch.float32).to(torch.bfloat16)
    step = torch.where(scale > 0, scale, 1.0).double()
    codes = ((g - low[..., None]) / step[..., None]).round().clamp(0, 15) * (scale > 0)[..., None]
    return codes.flatten(-2).to(torch.uint8), scale, low.to(torch.bfloat16) + 0.0


def _rows(k, v):
    """The cache rows [.., 144] of keys and values [.., 128]."""
    parts, numbers = [], []
    for x in (k, v):
        codes, scale, zero = _codes(x)
        parts.append(codes[..., 0::2] | codes[..., 1::2] << 4)
        numbers += [scale[..., 0], zero[..., 0], scale[..., 1], zero[..., 1]]
    return torch.cat([*parts, torch.stack(numbers, -1).contiguous().view(torch.uint8)], -1)


def _values(rows):
    """Keys and values [.., 128] that cache rows stand for, in 32 bits."""
    numbers = rows[..., 128:].contiguous().view(torch.bfloat16).float()
    out = []
    for i in range(2):
        b = rows[..., 64 * i:64 * i + 64]
        codes = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
        scale, zero = (numbers[..., [4 * i + j, 4 * i + 2 + j]].repeat_interleave(D // 2, -1) for j in (0, 1))
        out.append(codes * scale + zero)
    return out


def _places(s, total):
    """Sequence and cache position of every new token."""
    n, t = s["lens_k"].shape[0], torch.arange(total, device=s["lens_k"].device)
    cu = s["cu_q"] if s["cu_q"] is not None else torch.arange(n + 1, device=t.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, s["lens_k"][seq] - cu[seq + 1] + t


def _plain_append(s):
    rows = _rows(s["k"], s["v"])
    seq, at = _places(s, rows.shape[0])
    s["cache"][seq, at] = rows
    if s["k_out"] is None:
        return (s["cache"],)
    k, v = _values(rows)
    return s["cache"], k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_attn(s):
    q, len_k = s["q"], s["lens_k"]
    n, lq, lk = len_k.shape[0], s["max_q"], s["max_k"]
    cu = s["cu_q"] if s["cu_q"] is not None else torch.arange(n + 1, device=q.device)
    len_q = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + torch.arange(lq, device=q.device)).clamp(max=q.shape[0] - 1)
    kp, vp = _values(s["cache"][:, :lk])
    vp.masked_fill_((torch.arange(lk, device=q.device) >= len_k[:, None])[..., None, None], 0.0)
    hq, hk = q.shape[1], kp.shape[2]
    qp = q[rows].float().reshape(n, lq, hk, hq // hk, D).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, D)      # group's rows side by side
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
    t = torch.arange(q.shape[0], device=q.device)
    m = torch.searchsorted(cu[1:], t, right=True)
    out = o[m, t - cu[m]].to(torch.bfloat16)
    if s["lse"] is None:
        return (out,)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(n, lq, hq)
    return out, lse[m, t - cu[m]]


_plain = {"residual": _plain_residual, "gated": _plain_gated, "append": _plain_append, "attn": _plain_attn}


# ------------------------------ what a pass cannot do without ----------------------------------
SIZE = {"f32": 4, "bf16": 2}


def work(case):
    op = case["op"]
    if op == "residual":
        t, d = case["tokens"], case["dim"]
        weights = d * 4 * (2 if case["post"] else 1)
        gate = {"none": 0, "token": t * d * 2, "channel": d * 2}[case["gate"]]
        return {"bytes": t * d * (4 + 2 * SIZE[case["res"]]) + gate + weights, "flops": t * d * (6 + (4 if case["post"] else 0) + (case["gate"] != "none"))}
    if op == "gated":
        rows = case["tokens"] * case["h"]
        return {"bytes": rows * 3 * D * 2, "flops": rows * D * 9}
    lens_q, lens_k, hk = _ints(case["lens_q"]), _ints(case["lens_k"]), case["hk"]
    if op == "append":
        rows = sum(lens_q) * hk
        return {"bytes": rows * (4 * D + ROW + (4 * D if case["values"] else 0)), "flops": rows * 2 * D * 6}
    # query i of a sequence sees keys 0 .. i + lk - lq
    pairs = sum(lq * (lk - lq) + lq * (lq + 1) // 2 for lq, lk in zip(lens_q, lens_k))
    return {"bytes": sum(lens_q) * case["hq"] * (2 * D * 2 + (4 if case["lse"] else 0)) + sum(lens_k) * hk * ROW, "flops": 4 * D * case["hq"] * pairs}


# ------------------------------ the definition in 64 bits ---------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s, case)


def _exact_rms(x, weight):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()


def _exact_residual(s, case):
    u = s["y"].double()
    if case["post"]:
        u = _exact_rms(u, s["post_weight"])
    if case["gate"] != "none":
        u = u * s["gate"].double()
    r = s["residual"].double() + s["scale"] * u
    return r, _exact_rms(r, s["pre_weight"])


def _exact_gated(s, case):
    g = s["gate"].double()
    return _exact_rms(s["x"].double(), s["weight"]) * torch.sigmoid(g) * (g if case["silu"] else 1.0)


def _exact_append(s, case):
    cache, values = s["cache"].clone(), []
    place = [(n, lk - lq + i) for n, (lq, lk) in enumerate(zip(_ints(case["lens_q"]), _ints(case["lens_k"]))) for i in range(lq)]
    seq, at = torch.tensor(place, device=cache.device).T
    for which, x in enumerate((s["k"], s["v"])):
        value = []
        for half in range(2):
            g = x[..., 64 * half:64 * half + 64].double()
            zero, top = g.min(-1, keepdim=True)[0], g.max(-1, keepdim=True)[0]
            scale = ((top - zero) / 15).bfloat16().double()
            code = torch.zeros_like(g)
            for c in range(1, 16):         # borders that the value is above; on one, the even code of its two
                border = (c - 0.5) * scale
                code += ((g - zero > border) | ((g - zero == border) & (c % 2 == 0))) & (scale > 0)
            value.append(code * scale + zero)
            both = code.reshape(*code.shape[:-1], 32, 2)
            cache[seq, at, :, 64 * which + 32 * half:64 * which + 32 * half + 32] = (both[..., 0] + 16 * both[..., 1]).to(torch.uint8)
            numbers = torch.cat([scale, zero + 0.0], -1).bfloat16().view(torch.uint8)
            cache[seq, at, :, 128 + 8 * which + 4 * half:132 + 8 * which + 4 * half] = numbers
        values.append(torch.cat(value, -1))
    return (cache, *values) if case["values"] else (cache,)


def _exact_attn(s, case):
    lens_q, lens_k = _ints(case["lens_q"]), _ints(case["lens_k"])
    q, hq, hk = s["q"], case["hq"], case["hk"]
    out = torch.zeros(q.shape, device=q.device, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], device=q.device, dtype=torch.float64)
    shift = torch.tensor([0, 4], device=q.device)
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        for h in range(hk):
            rows = s["cache"][n, :lk, h].contiguous()
            codes = (rows[:, :128, None].long() >> shift & 15).reshape(lk, 2, 2, 64).double()          # key or value, half, channel
            scale, zero = rows[:, 128:].contiguous().view(torch.bfloat16).double().reshape(lk, 2, 2, 2).unbind(-1)
            kh, vh = (codes * scale[..., None] + zero[..., None]).flatten(2).unbind(1)
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


_exact = {"residual": _exact_residual, "gated": _exact_gated, "append": _exact_append, "attn": _exact_attn}
