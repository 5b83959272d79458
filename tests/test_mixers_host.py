"""Host checks of the token mixers' C ABI (no GPU): requests that contradict themselves are
refused with the right status before anything is enqueued, so the addresses are fake and
never dereferenced."""
import ctypes

import pytest
import torch

from gated_delta_rule_36_gb300 import binding as kb
from gated_delta_rule_36_gb300 import build as kbuild

BASE = 0x7F0000000000
MB = 1 << 20
BF, F32, I64 = kb.KDA_BF16, kb.KDA_F32, kb.KDA_I64
INVALID, UNSUPPORTED, ALIAS, WORKSPACE = (kb.KDA_ERR_INVALID_ARG, kb.KDA_ERR_UNSUPPORTED, kb.KDA_ERR_ALIAS,
                                          kb.KDA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kb.load()


def view(shape, at, stride=None, dtype=BF):
    """A packed kda_view (contiguous unless strides are given) at BASE + at."""
    if stride is None:
        stride, n = [], 1
        for s in reversed(shape):
            stride.insert(0, n)
            n *= s
    pad = kb._PAD[len(shape)]
    return kb._PACK_VIEW(BASE + at, dtype, len(shape), *shape, *pad, *stride, *pad)


def dense(shape, at, dtype=F32):
    return kb._PACK_DENSE(BASE + at, dtype, len(shape), *shape, *kb._PAD[len(shape)])


def test_view_bytes_match_the_header_struct():
    class View(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                    ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]
    v = View.from_buffer_copy(view((5, 3, 128), 64, (1280, 256, 1), F32))
    assert ctypes.sizeof(View) == len(view((1,), 0)) and ctypes.sizeof(kb.KdaTensor) == len(dense((1,), 0))
    assert (v.data, v.dtype, v.ndim, list(v.shape), list(v.stride)) == (BASE + 64, F32, 3, [5, 3, 128, 0], [1280, 256, 1, 0])


# ------------------------------------------------------------------ norm and rotation
T, HQ, HK = 6, 4, 2


def rope(lib, **over):
    a = dict(q=view((T, HQ, 128), 0), k=view((T, HK, 128), MB), qw=dense((128,), 2 * MB), kw=dense((128,), 3 * MB), eps=1e-6,
             cs=dense((100, 64), 4 * MB), pos=dense((T,), 5 * MB, I64), qo=view((T, HQ, 128), 6 * MB), ko=view((T, HK, 128), 7 * MB),
             status=None, flags=0)
    a.update(over)
    return lib.kda_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["eps"], a["cs"], a["pos"], a["qo"], a["ko"], a["status"],
                                a["flags"], None)


ROPE = [
    (dict(flags=2), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(status=BASE + 2), INVALID),
    (dict(q=None), INVALID),
    (dict(k=None), INVALID),                                              # k_out without k
    (dict(q=view((T, HQ, 64), 0)), UNSUPPORTED),
    (dict(q=view((T, HQ, 128), 0, dtype=F32)), INVALID),
    (dict(q=view((T, HQ, 128), 8)), INVALID),                             # 16-byte alignment
    (dict(q=view((T, HQ, 128), 0, (HQ * 128, 128, 2))), INVALID),         # innermost stride
    (dict(q=view((T, HQ, 128), 0, (HQ * 128 + 4, 128, 1))), INVALID),     # stride not a multiple of 8
    (dict(q=view((T, HQ, 128), 0, (0, 128, 1))), INVALID),                # broadcast rows
    (dict(q=view((T, HQ, 128), 0, (HQ * 128, 64, 1))), INVALID),          # heads that overlap
    (dict(k=view((T + 1, HK, 128), MB)), INVALID),
    (dict(qo=view((T, HQ + 1, 128), 6 * MB)), INVALID),
    (dict(qw=dense((64,), 2 * MB)), INVALID),
    (dict(qw=dense((128,), 2 * MB, I64)), INVALID),
    (dict(pos=None), INVALID),
    (dict(cs=None), INVALID),
    (dict(cs=dense((100, 24), 4 * MB)), UNSUPPORTED),
    (dict(cs=dense((100, 144), 4 * MB)), UNSUPPORTED),
    (dict(cs=dense((100,), 4 * MB)), INVALID),
    (dict(pos=dense((T + 1,), 5 * MB, I64)), INVALID),
    (dict(pos=dense((T,), 5 * MB, F32)), INVALID),
    (dict(qo=view((T, HQ, 128), 256)), ALIAS),                            # q shifted by one head
    (dict(qo=view((T, HK, 128), MB), q=view((T, HK, 128), 0)), ALIAS),    # q_out is k
    (dict(ko=view((T, HK, 128), 6 * MB + 128)), ALIAS),                   # k_out meets q_out
    (dict(qo=view((T, HQ, 128), 4 * MB)), ALIAS),                         # q_out over the table
]


@pytest.mark.parametrize("over,expect", ROPE, ids=range(len(ROPE)))
def test_norm_rope_refusals(lib, over, expect):
    assert rope(lib, **over) == expect
    assert lib.kda_last_error()


# ------------------------------------------------------------------ attention
def attn(lib, **over):
    n = 2
    a = dict(q=view((T, HQ, 128), 0), k=view((T, HK, 128), MB), v=view((T, HK, 128), 2 * MB), scale=0.1, out=view((T, HQ, 128), 3 * MB),
             lse=None, cuq=dense((n + 1,), 4 * MB, I64), cuk=None, lens=None, ws=BASE + 8 * MB, nb=1 << 40)
    a.update(over)
    return lib.kda_attn_fwd(a["q"], a["k"], a["v"], a["scale"], a["out"], a["lse"], a["cuq"], a["cuk"], a["lens"], a["ws"], a["nb"], None)


CACHE = dict(k=view((2, 50, HK, 128), MB), v=view((2, 50, HK, 128), 2 * MB), lens=dense((2,), 5 * MB, I64))
ATTN = [
    (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID),
    (dict(q=view((T, HQ, 64), 0)), UNSUPPORTED),
    (dict(k=view((T, HK, 64), MB)), UNSUPPORTED),
    (dict(k=view((T, 3, 128), MB)), INVALID),                             # 3 does not divide 4
    (dict(q=view((T, 258, 128), 0), k=view((T, 2, 128), MB)), UNSUPPORTED),   # 129 heads in a group
    (dict(v=view((T, HQ, 128), 2 * MB)), INVALID),
    (dict(v=None), INVALID),
    (dict(k=view((T + 1, HK, 128), MB), v=view((T + 1, HK, 128), 2 * MB)), INVALID),   # no cu_seqlens_k: Tk must be Tq
    (dict(cuq=dense((3,), 4 * MB, F32)), INVALID),
    (dict(cuk=dense((4,), 5 * MB, I64)), INVALID),                        # another number of sequences
    (dict(cuq=None, cuk=dense((5,), 5 * MB, I64)), INVALID),              # 6 queries over 4 sequences
    (dict(lens=dense((2,), 5 * MB, I64)), INVALID),                       # lengths without a cache
    (dict(CACHE, lens=None), INVALID),
    (dict(CACHE, cuk=dense((3,), 6 * MB, I64)), INVALID),
    (dict(CACHE, lens=dense((3,), 5 * MB, I64)), INVALID),
    (dict(CACHE, v=view((2, 51, HK, 128), 2 * MB)), INVALID),
    (dict(CACHE, cuq=dense((4,), 4 * MB, I64)), INVALID),                 # three sequences, a cache of two
    (dict(CACHE, cuq=None, q=view((5, HQ, 128), 0), out=view((5, HQ, 128), 3 * MB)), INVALID),
    (dict(lse=dense((T, HK), 6 * MB)), INVALID),
    (dict(lse=dense((T, HQ), 6 * MB, I64)), INVALID),
    (dict(out=view((T, HQ, 128), 0)), ALIAS),
    (dict(out=view((T, HQ, 128), 2 * MB + 256)), ALIAS),
    (dict(lse=dense((T, HQ), 3 * MB)), ALIAS),
    (dict(lse=dense((T, HQ), 4 * MB)), ALIAS),
    (dict(ws=0), WORKSPACE),
    (dict(ws=BASE + 8 * MB + 16), WORKSPACE),
    (dict(nb=255), WORKSPACE),
]


@pytest.mark.parametrize("over,expect", ATTN, ids=range(len(ATTN)))
def test_attn_refusals(lib, over, expect):
    assert attn(lib, **over) == expect
    assert lib.kda_last_error()


def test_attn_workspace_size(lib):
    assert kb.kda_attn_workspace_size(1, 32, 8) >= 256
    assert kb.kda_attn_workspace_size(-1, 32, 8) == 0
    assert kb.kda_attn_workspace_size(1, 32, 5) == 0


# ------------------------------------------------------------------ linear attention
H = 3


def lin(lib, **over):
    a = dict(q=view((1, T, H, 128), 0), k=view((1, T, H, 128), MB), v=view((1, T, H, 128), 2 * MB), ld=dense((H,), 3 * MB), scale=0.1,
             out=view((1, T, H, 128), 4 * MB), init=None, final=None, cu=None, ws=BASE + 64 * MB, nb=1 << 40)
    a.update(over)
    return lib.kda_lin_fwd(a["q"], a["k"], a["v"], a["ld"], a["scale"], a["out"], a["init"], a["final"], a["cu"], a["ws"], a["nb"], None)


STATE = (1, H, 128, 128)
LIN = [
    (dict(scale=float("nan")), INVALID),
    (dict(q=view((T, H, 128), 0)), INVALID),
    (dict(q=view((1, T, H, 64), 0)), UNSUPPORTED),
    (dict(k=view((1, T, H + 1, 128), MB)), INVALID),
    (dict(q=view((2, 3, H, 128), 0, (4 * H * 128, H * 128, 128, 1)), k=view((2, 3, H, 128), MB), v=view((2, 3, H, 128), 2 * MB),
          out=view((2, 3, H, 128), 4 * MB)), INVALID),                    # batch rows apart
    (dict(ld=dense((H + 1,), 3 * MB)), INVALID),
    (dict(ld=None), INVALID),
    (dict(init=dense((1, H, 128, 64), 8 * MB)), INVALID),
    (dict(final=dense(STATE, 8 * MB, I64)), INVALID),
    (dict(init=dense(STATE, 8 * MB), final=dense(STATE, 8 * MB + 4096)), ALIAS),
    (dict(init=dense(STATE, 8 * MB), final=dense(STATE, 8 * MB, BF)), ALIAS),
    (dict(final=dense(STATE, 2 * MB)), ALIAS),
    (dict(out=view((1, T, H, 128), 2 * MB)), ALIAS),
    (dict(out=view((1, T, H, 128), 3 * MB)), ALIAS),
    (dict(cu=dense((3,), 8 * MB, F32)), INVALID),
    (dict(cu=dense((3,), 8 * MB, I64), init=dense(STATE, 9 * MB)), INVALID),   # two sequences, one state
    (dict(q=view((2, 3, H, 128), 0), k=view((2, 3, H, 128), MB), v=view((2, 3, H, 128), 2 * MB), out=view((2, 3, H, 128), 4 * MB),
          cu=dense((3,), 8 * MB, I64)), INVALID),                         # packed mode has B == 1
    (dict(ws=0), WORKSPACE),
    (dict(nb=128), WORKSPACE),
]


@pytest.mark.parametrize("over,expect", LIN, ids=range(len(LIN)))
def test_lin_fwd_refusals(lib, over, expect):
    assert lin(lib, **over) == expect
    assert lib.kda_last_error()


def step(lib, **over):
    B = 2
    a = dict(q=view((B, H, 128), 0), k=view((B, H, 128), MB), v=view((B, H, 128), 2 * MB), ld=dense((H,), 3 * MB), scale=0.1,
             out=view((B, H, 128), 4 * MB), init=None, final=None)
    a.update(over)
    return lib.kda_lin_decode(a["q"], a["k"], a["v"], a["ld"], a["scale"], a["out"], a["init"], a["final"], None)


STATE2 = (2, H, 128, 128)
STEP = [
    (dict(scale=float("inf")), INVALID),
    (dict(q=view((2, H, 96), 0)), UNSUPPORTED),
    (dict(v=view((2, H, 128), 2 * MB, (H * 128 + 2, 128, 1))), INVALID),
    (dict(ld=dense((H,), 3 * MB, I64)), INVALID),
    (dict(init=dense(STATE, 8 * MB)), INVALID),
    (dict(init=dense(STATE2, 8 * MB), final=dense(STATE2, 8 * MB + 65536)), ALIAS),
    (dict(out=view((2, H, 128), MB)), ALIAS),
    (dict(final=dense(STATE2, 0)), ALIAS),
]


@pytest.mark.parametrize("over,expect", STEP, ids=range(len(STEP)))
def test_lin_decode_refusals(lib, over, expect):
    assert step(lib, **over) == expect
    assert lib.kda_last_error()


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    for call in (lambda t: kb.kda_lin_decode(t, x, x, torch.zeros(2), 1.0, x), lambda t: kb.kda_attn_fwd(t, x, x, 1.0, x),
                 lambda t: kb.kda_qk_norm_rope(t, None, None, None, None, None, x, None)):
        with pytest.raises(ValueError):
            call(x)
        with pytest.raises(TypeError):
            call("q")
