"""Linear attention prompts whose state is updated in place: outputs and states are, bit for bit, those of a
call with two buffers, which are checked against 64 bits (the bounds of test_gpu_mixers.py).  The
units lie in one, two and more shares of the SMs; in the latter case the share that begins a unit may come
to it in its main pass long after the last one has written the final state.
"""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import D, LINS, NAN, check_lin_out, check_state, cu_of, gen_of, rand
from test_gpu_mixers_shapes import DIVIDED, chunked_lin

pytestmark = pytest.mark.gpu

LONG = [([8192], 32), ([8192], 64), ([32768], 32), ([4096], 40), ([12000], 40), ([5000, 0, 9000], 12)]


def two_buffers_then_one(lens, h, dtype, repeats):
    g = gen_of(sum(lens) + h)
    q, k, v = (rand(g, 1, sum(lens), h, D) for _ in range(3))
    ld = -(2.0 ** (-10.0 * torch.arange(1, h + 1) / h)).cuda()
    init, final = rand(g, len(lens), h, D, D, dtype=dtype), torch.full((len(lens), h, D, D), NAN, dtype=dtype, device="cuda")
    out = torch.full_like(q, NAN)
    cu = cu_of(lens)
    ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, out, initial_state=init, final_state=final, cu_seqlens=cu)
    assert kda.kda_read_device_status(ws) == 0
    for _ in range(repeats):
        state, again = init.clone(), torch.full_like(q, NAN)
        ws = kda.kda_lin_fwd(q, k, v, ld, 0.1, again, initial_state=state, final_state=state, cu_seqlens=cu)
        assert kda.kda_read_device_status(ws) == 0
        assert torch.equal(again, out) and torch.equal(state, final)
    if sum(lens):
        o, A, s, t = chunked_lin(q[0], k[0], v[0], ld, 0.1, lens, init)
        check_lin_out(out[0], o, A)
        check_state("final_state", final, s, t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,h", LONG, ids=[f"{'-'.join(map(str, a))}x{b}" for a, b in LONG])
def test_long_prompts_in_place(lens, h, dtype):
    two_buffers_then_one(lens, h, dtype, 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,h", DIVIDED + LINS, ids=[f"{'-'.join(map(str, a))}x{b}" for a, b in DIVIDED + LINS])
def test_any_division_in_place(lens, h, dtype):
    two_buffers_then_one(lens, h, dtype, 2)


def test_a_prompt_in_parts_is_the_whole_prompt():
    """One state pool carried from part to part of two prompts, as a server does."""
    g = gen_of(77)
    h, parts = 24, ([2100, 700], [1, 1300], [4000, 129])
    total = [sum(p[n] for p in parts) for n in range(2)]
    q, k, v = (rand(g, 2, max(total), h, D) for _ in range(3))
    ld = -(2.0 ** (-10.0 * torch.arange(1, h + 1) / h)).cuda()
    state = rand(g, 2, h, D, D, dtype=torch.float32)
    init, out, at = state.clone(), torch.full_like(q, NAN), [0, 0]
    for lens in parts:
        cut = lambda x: torch.cat([x[n, at[n]:at[n] + lens[n]] for n in range(2)])[None]
        o = torch.full_like(cut(q), NAN)
        ws = kda.kda_lin_fwd(cut(q), cut(k), cut(v), ld, 0.1, o, initial_state=state, final_state=state, cu_seqlens=cu_of(lens))
        assert kda.kda_read_device_status(ws) == 0
        for n, piece in enumerate(o[0].split(lens)):
            out[n, at[n]:at[n] + lens[n]] = piece
            at[n] += lens[n]
    join = lambda x: torch.cat([x[n, :total[n]] for n in range(2)])
    o, A, s, t = chunked_lin(join(q), join(k), join(v), ld, 0.1, total, init)
    check_lin_out(join(out), o, A)
    check_state("state", state, s, t)
