"""The mixers on parts of one buffer that lie between one another: inputs and output are columns of a
projection, heads in turn or planes; the bits are those of calls on buffers of their own, and what lies
between the parts is not touched.
"""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import D, cu_of, gen_of, rand, table

pytestmark = pytest.mark.gpu
T, H = 333, 6
LAYOUTS = {   # shape of the buffer and its parts as [T, H, 128]
    "columns": ((T, 5, H, D), lambda b, i: b[:, i]), "heads_in_turn": ((T, H, 5, D), lambda b, i: b[:, :, i]),
    "planes": ((5, T, H, D), lambda b, i: b[i]), "heads_outside": ((H, T, 5, D), lambda b, i: b[:, :, i].transpose(0, 1)),
}


def parts(name, seed):
    shape, of = LAYOUTS[name]
    buf = rand(gen_of(seed), *shape)
    views = [of(buf, i) for i in range(5)]
    return buf, views, [v.contiguous() for v in views]


@pytest.mark.parametrize("name", LAYOUTS)
def test_norm_rope_in_place(name):
    buf, (q, k, v, a, b), (cq, ck, cv, ca, cb) = parts(name, 81)
    cs, pos = table(500, 128), torch.arange(T, device="cuda")
    oq, ok = torch.empty_like(cq), torch.empty_like(ck)
    kda.kda_qk_norm_rope(cq, ck, None, None, cs, pos, oq, ok)
    kda.kda_qk_norm_rope(q, k, None, None, cs, pos, q, k)                    # in place
    assert torch.equal(q, oq) and torch.equal(k, ok)
    kda.kda_qk_norm_rope(v, None, None, None, cs, pos, b, None)              # into another part
    kda.kda_qk_norm_rope(cv, None, None, None, cs, pos, oq, None)
    assert torch.equal(b, oq) and torch.equal(a, ca) and torch.equal(v, cv)


@pytest.mark.parametrize("name", LAYOUTS)
def test_attn_and_lin(name):
    buf, (q, k, v, out, rest), (cq, ck, cv, _, crest) = parts(name, 82)
    cu, want = cu_of([200, 133]), torch.empty_like(cq)
    kda.kda_attn_fwd(cq, ck, cv, 0.1, want, cu_seqlens_q=cu)
    ws = kda.kda_attn_fwd(q, k, v, 0.1, out, cu_seqlens_q=cu)
    assert kda.kda_read_device_status(ws) == 0 and torch.equal(out, want)
    ld = torch.full((H,), -0.1, device="cuda")
    kda.kda_lin_fwd(cq[None], ck[None], cv[None], ld, 0.1, want[None], cu_seqlens=cu)
    ws = kda.kda_lin_fwd(q[None], k[None], v[None], ld, 0.1, out[None], cu_seqlens=cu)
    assert kda.kda_read_device_status(ws) == 0 and torch.equal(out, want)
    kda.kda_lin_decode(cq, ck, cv, ld, 0.1, want)
    kda.kda_lin_decode(q, k, v, ld, 0.1, out)
    assert torch.equal(out, want)
    assert torch.equal(rest, crest) and torch.equal(q, cq) and torch.equal(k, ck) and torch.equal(v, cv)
