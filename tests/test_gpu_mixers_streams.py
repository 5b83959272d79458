"""A workspace that the mixers' binding allocates belongs to the stream that the call is put on: memory
that was just freed on the current stream may still be in use there, so a call on another stream must not get it.
"""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import D, NAN, cu_of, gen_of, rand

pytestmark = pytest.mark.gpu


def calls():
    g = gen_of(71)
    q, k, v = (rand(g, 300, 4, D) for _ in range(3))
    ld, cu = torch.full((4,), -0.1, device="cuda"), cu_of([200, 100])
    nbytes = {"attn": kda.kda_attn_workspace_size(300, 4, 4), "lin": kda.kda_lin_workspace_size(300, 4, 2)}
    return nbytes, {"attn": lambda out, **kw: kda.kda_attn_fwd(q, k, v, 0.1, out, cu_seqlens_q=cu, **kw),
                    "lin": lambda out, **kw: kda.kda_lin_fwd(q[None], k[None], v[None], ld, 0.1, out[None], cu_seqlens=cu, **kw)}


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", ["attn", "lin"])
def test_workspace_is_not_memory_just_freed_on_another_stream(name, how):
    nbytes, call = calls()
    want, out = (torch.full((300, 4, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call[name](want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = torch.empty(nbytes[name], dtype=torch.uint8, device="cuda")
    first, last = freed.data_ptr(), freed.data_ptr() + freed.numel()
    del freed
    ws = call[name](out, stream=s if how == "stream" else s.cuda_stream)
    assert ws.data_ptr() >= last or ws.data_ptr() + ws.numel() <= first
    assert kda.kda_read_device_status(ws, stream=s) == 0
    assert torch.equal(out, want)
    # and given back, it goes to the next call on that stream, not to the current one
    at = ws.data_ptr()
    del ws
    other = torch.empty(nbytes[name], dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != at
    torch.cuda.synchronize()
