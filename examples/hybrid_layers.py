"""Three token mixers in one small model: prompts, then single tokens.

    python examples/hybrid_layers.py

The model is a stack of residual layers x + W_out mix(norm(x) W_in) whose mixers are KDA, linear attention
with a decay for each head, and grouped-head softmax attention, as hybrid models interleave them (random
weights; no feed-forward layers, which are plain matrix products).  A layer's queries, keys and values are
columns of one projection, which the mixers read as strided views:

  attention   kda_qk_norm_rope on the queries and keys in place, the keys and values into the
              cache, kda_attn_fwd (packed prompts; later the cache, one token a sequence)
  linear      kda_qk_norm_rope without a rotation, kda_lin_fwd / kda_lin_decode on an fp32 state
  kda         kda_fwd / kda_decode on an fp32 state

The check runs the prompts and then some steps, and compares with one run over the longer prompts.
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_36_gb300 as kda

D = 128


class Cache:
    """What the sequences keep between calls: one entry for each layer."""

    def __init__(self, model, nseq, room):
        dev, H, Hk = "cuda", model.heads, model.kv_heads
        self.lens = torch.zeros(nseq, dtype=torch.int64, device=dev)
        self.layers = [torch.zeros(2, nseq, room, Hk, D, dtype=torch.bfloat16, device=dev) if kind == "attention" else
                       torch.zeros(nseq, H, D, D, device=dev) for kind in model.kinds]


class Model:
    def __init__(self, kinds=("kda", "linear", "attention"), hidden=256, heads=6, kv_heads=2, reach=4096, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kinds, self.heads, self.kv_heads = kinds, heads, kv_heads
        rand = lambda *shape, mul: (torch.randn(shape, generator=g) * mul).cuda()
        columns = {"kda": 4 * heads * D + heads, "linear": 3 * heads * D, "attention": (heads + 2 * kv_heads) * D}
        self.w_in = [rand(hidden, columns[k], mul=hidden ** -0.5).bfloat16() for k in kinds]
        self.w_out = [rand(heads * D, hidden, mul=(heads * D) ** -0.5).bfloat16() for _ in kinds]
        self.q_weight, self.k_weight = 1 + rand(D, mul=0.1), 1 + rand(D, mul=0.1)
        self.A_log, self.dt_bias = rand(heads, mul=0.5), rand(heads, D, mul=0.5)
        self.log_decay = -(2.0 ** (-8.0 * torch.arange(1, heads + 1) / heads)).cuda()
        angle = torch.arange(reach)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def forward(self, x, cache, cu_seqlens=None):
        """x [T, hidden]: packed prompts of new sequences with cu_seqlens, else one token for each sequence."""
        nseq, H, Hk, T = cache.lens.numel(), self.heads, self.kv_heads, x.shape[0]
        if cu_seqlens is None:
            seq, pos = torch.arange(nseq, device="cuda"), cache.lens
        else:
            seq = torch.repeat_interleave(torch.arange(nseq, device="cuda"), cu_seqlens.diff(), output_size=T)
            pos = torch.arange(T, device="cuda") - cu_seqlens[seq]
        scale, statuses = D ** -0.5, []
        for kind, w_in, w_out, kept in zip(self.kinds, self.w_in, self.w_out, cache.layers):
            y = torch.nn.functional.rms_norm(x, x.shape[1:]).bfloat16() @ w_in
            out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
            if kind == "attention":
                q, k, v = (t.unflatten(1, (-1, D)) for t in y.split([H * D, Hk * D, Hk * D], 1))
                rope_status = torch.zeros(4, dtype=torch.uint8, device="cuda")
                kda.kda_qk_norm_rope(q, k, self.q_weight, self.k_weight, self.cos_sin, pos, q, k, status=rope_status)
                kept[0, seq, pos], kept[1, seq, pos] = k, v
                if cu_seqlens is None:
                    ws = kda.kda_attn_fwd(q, kept[0], kept[1], scale, out, seqlens_k=cache.lens + 1)
                else:
                    ws = kda.kda_attn_fwd(q, k, v, scale, out, cu_seqlens_q=cu_seqlens)
                statuses += [rope_status, ws]
            elif kind == "linear":
                q, k, v = (t.unflatten(1, (H, D)) for t in y.split(H * D, 1))
                kda.kda_qk_norm_rope(q, k, self.q_weight, self.k_weight, None, None, q, k)
                if cu_seqlens is None:
                    kda.kda_lin_decode(q, k, v, self.log_decay, scale / D, out, initial_state=kept, final_state=kept)
                else:
                    statuses.append(kda.kda_lin_fwd(q[None], k[None], v[None], self.log_decay, scale / D, out[None],
                                                    final_state=kept, cu_seqlens=cu_seqlens))
            else:
                q, k, v, gate = (t.unflatten(1, (H, D)).contiguous() for t in y[:, :4 * H * D].split(H * D, 1))
                beta = y[:, 4 * H * D:].sigmoid().contiguous()
                args = (self.A_log, self.dt_bias, -5.0)
                if cu_seqlens is None:
                    kda.kda_decode(q, k, v, gate, beta, scale, out, *args, initial_state=kept, final_state=kept)
                else:
                    statuses.append(kda.kda_fwd(*(t[None] for t in (q, k, v, gate, beta)), scale, out[None], *args,
                                                final_state=kept, cu_seqlens=cu_seqlens))
            x = x + (out.flatten(1) @ w_out).float()
        cache.lens += 1 if cu_seqlens is None else cu_seqlens.diff()
        bits = [kda.kda_read_device_status(s) for s in statuses]
        if any(bits):
            raise RuntimeError(f"device status bits {bits}")
        return x


def check(lens=(37, 1, 200, 130), steps=5, hidden=256):
    """Relative difference (Frobenius) between prompts followed by single tokens and the longer prompts."""
    model = Model(hidden=hidden)
    cu = lambda ls: torch.tensor([0, *ls], dtype=torch.int64).cumsum(0).cuda()
    g = torch.Generator().manual_seed(1)
    longer = [n + steps for n in lens]
    at = [0] + torch.tensor(longer).cumsum(0).tolist()
    x = torch.randn(sum(longer), hidden, generator=g).cuda()
    whole = model.forward(x, Cache(model, len(lens), max(longer)), cu(longer))
    cache = Cache(model, len(lens), max(longer))
    rows = torch.cat([torch.arange(at[n], at[n] + lens[n]) for n in range(len(lens))]).cuda()
    parts, order = [model.forward(x[rows], cache, cu(lens))], [rows]
    for i in range(steps):
        rows = torch.tensor([at[n] + lens[n] + i for n in range(len(lens))], device="cuda")
        parts.append(model.forward(x[rows], cache))
        order.append(rows)
    got = torch.empty_like(whole)
    got[torch.cat(order)] = torch.cat(parts)
    return ((got - whole).norm() / whole.norm()).item()


if __name__ == "__main__":
    print(f"prompts and steps against longer prompts: relative difference {check():.2e}")
