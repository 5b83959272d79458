"""Host checks of the operators around the mixers (no GPU): requests that contradict themselves are refused
with the right status before anything is enqueued, so the addresses are fake and never dereferenced."""
import pytest
import torch

from gated_delta_rule_36_gb300 import binding as kb
from test_mixers_devices import D, Library, On0, On1, tensors, ws
from test_mixers_host import ALIAS, BASE, BF, F32, I64, INVALID, MB, UNSUPPORTED, WORKSPACE, dense, lib, view  # noqa: F401

U8, ROW = kb.KDA_U8, 144
T, HQ, HK, N, S = 6, 8, 2, 3, 50
NAN = float("nan")
CACHE = (N, S, HK, ROW)


def cache(shape=CACHE, at=20 * MB, stride=None, dtype=U8):
    return view(shape, at, stride, dtype)


# ------------------------------------------------------------------ append
def append(lib, **over):
    a = dict(k=view((T, HK, 128), 0), v=view((T, HK, 128), MB), cache=cache(), lens=dense((N,), 2 * MB, I64), cu=dense((N + 1,), 3 * MB, I64),
             ko=None, vo=None, status=None)
    a.update(over)
    return lib.kda_qcache_append(a["k"], a["v"], a["cache"], a["lens"], a["cu"], a["ko"], a["vo"], a["status"], None)


OUT = dict(ko=view((T, HK, 128), 4 * MB), vo=view((T, HK, 128), 5 * MB))
APPEND = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(lens=None), INVALID),
    (dict(k=view((T, HK, 64), 0)), UNSUPPORTED), (dict(k=view((T, HK, 128), 0, dtype=F32)), INVALID), (dict(k=view((T * HK, 128), 0)), INVALID),
    (dict(v=view((T + 1, HK, 128), MB)), INVALID), (dict(v=view((T, HK, 128), MB + 8)), INVALID), (dict(v=view((T, HK, 128), MB, (4 * 128, 128, 2))), INVALID),
    (dict(status=BASE + 2), INVALID),
    (dict(cache=cache(dtype=BF)), INVALID), (dict(cache=cache((N, S, HK, 128))), INVALID), (dict(cache=view((S, HK, ROW), 20 * MB, dtype=U8)), INVALID),
    (dict(cache=cache((N + 1, S, HK, ROW))), INVALID), (dict(cache=cache((N, S, HK + 1, ROW))), INVALID), (dict(cache=cache(at=20 * MB + 8)), INVALID),
    (dict(cache=cache(stride=(S * HK * ROW, HK * ROW, ROW, 2))), INVALID), (dict(cache=cache(stride=(S * HK * ROW, HK * ROW + 8, ROW, 1))), INVALID),
    (dict(cache=cache(stride=(S * HK * ROW, HK * ROW, 128, 1))), INVALID), (dict(cache=cache(stride=(0, HK * ROW, ROW, 1))), INVALID),
    (dict(cache=cache((N, (1 << 30) + 1, HK, ROW))), UNSUPPORTED), (dict(cache=cache(stride=(1 << 47, HK * ROW, ROW, 1))), INVALID),
    (dict(lens=dense((N + 1,), 2 * MB, I64)), INVALID), (dict(lens=dense((N,), 2 * MB)), INVALID), (dict(cu=dense((N,), 3 * MB, I64)), INVALID),
    (dict(cu=dense((2, 2), 3 * MB, I64)), INVALID), (dict(cu=dense((N + 1,), 3 * MB + 4, I64)), INVALID),
    (dict(cu=None, k=view((T + 1, HK, 128), 0), v=view((T + 1, HK, 128), MB)), INVALID),                       # tokens that do not divide
    (dict(cu=None, cache=cache((0, S, HK, ROW)), lens=dense((0,), 2 * MB, I64)), INVALID),                      # tokens without a sequence
    (dict(cu=dense((40001,), 3 * MB, I64), cache=cache((40000, S, HK, ROW)), lens=dense((40000,), 2 * MB, I64)), UNSUPPORTED),
    (dict(k=view(((1 << 30) + 1, HK, 128), 0), v=view(((1 << 30) + 1, HK, 128), 1 << 44)), UNSUPPORTED),
    (dict(ko=OUT["ko"]), INVALID), (dict(vo=OUT["vo"]), INVALID), (dict(OUT, ko=view((T, HK, 128), 4 * MB, dtype=F32)), INVALID),
    (dict(OUT, ko=view((T, HK, 128), MB)), ALIAS),                                                              # k_out is v
    (dict(OUT, vo=view((T, HK, 128), 0)), ALIAS),
    (dict(OUT, ko=view((T, HK, 128), 256)), ALIAS),                                                             # k shifted
    (dict(OUT, vo=OUT["ko"]), ALIAS), (dict(OUT, ko=view((T, HK, 128), 20 * MB)), ALIAS), (dict(cache=cache(at=0)), ALIAS), (dict(cache=cache(at=MB)), ALIAS),
    (dict(cache=cache(stride=(ROW, HK * ROW, ROW, 1))), ALIAS), (dict(cache=cache(stride=(S * HK * ROW, ROW, ROW, 1))), ALIAS),      # rows on one another
    (dict(OUT, ko=view((T, HK, 128), 4 * MB, (128, 128, 1))), ALIAS),
    (dict(cache=cache(at=2 * MB - 1024)), ALIAS), (dict(cache=cache(at=3 * MB - 1024)), ALIAS), (dict(OUT, vo=view((T, HK, 128), 2 * MB - 256)), ALIAS),
]


@pytest.mark.parametrize("over,want", APPEND)
def test_append_refusals(lib, over, want):  # noqa: F811
    assert append(lib, **over) == want
    assert lib.kda_last_error()


# ------------------------------------------------------------------ attention
def attn(lib, **over):
    a = dict(q=view((T, HQ, 128), 0), cache=cache(), scale=0.1, out=view((T, HQ, 128), MB), lens=dense((N,), 2 * MB, I64), lse=dense((T, HQ), 4 * MB),
             cu=dense((N + 1,), 3 * MB, I64), ws=BASE + 64 * MB, nbytes=256 * MB)
    a.update(over)
    return lib.kda_attn_qcache_fwd(a["q"], a["cache"], a["scale"], a["out"], a["lens"], a["lse"], a["cu"], a["ws"], a["nbytes"], None)


ATTN = [
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(out=None), INVALID), (dict(lens=None), INVALID),
    (dict(q=view((T, HQ, 64), 0)), UNSUPPORTED), (dict(q=view((T, HQ, 128), 0, dtype=F32)), INVALID), (dict(q=view((T, 5, 128), 0)), INVALID),
    (dict(q=view((T, 2 * 129, 128), 0), out=view((T, 2 * 129, 128), 8 * MB), lse=None), UNSUPPORTED),
    (dict(q=view((T, HQ, 128), 0, (HQ * 128, 64, 1))), INVALID), (dict(out=view((T + 1, HQ, 128), MB)), INVALID),
    (dict(cache=cache(dtype=I64)), INVALID), (dict(cache=cache((N, S, HK, 143))), INVALID), (dict(cache=cache((N, S, 0, ROW))), INVALID),
    (dict(cache=cache((N - 1, S, HK, ROW))), INVALID), (dict(cache=cache(at=20 * MB + 4)), INVALID), (dict(cache=cache(stride=(S * HK * ROW, HK * ROW, 136, 1))), INVALID),
    (dict(cache=cache(stride=(S * HK * ROW, ROW, S * ROW + 8, 1))), INVALID),
    (dict(lens=dense((N - 1,), 2 * MB, I64)), INVALID), (dict(cu=dense((N + 2,), 3 * MB, I64)), INVALID), (dict(cu=dense((N + 1,), 3 * MB)), INVALID),
    (dict(cu=None, q=view((T + 1, HQ, 128), 0), out=view((T + 1, HQ, 128), MB), lse=None), INVALID),
    (dict(lse=dense((T, HQ + 1), 4 * MB)), INVALID), (dict(lse=dense((T, HQ), 4 * MB, BF)), INVALID),
    (dict(out=view((T, HQ, 128), 0)), ALIAS), (dict(out=view((T, HQ, 128), 20 * MB)), ALIAS), (dict(out=view((T, HQ, 128), 2 * MB - 256)), ALIAS),
    (dict(out=view((T, HQ, 128), 3 * MB - 256)), ALIAS), (dict(out=view((T, HQ, 128), 4 * MB - 256)), ALIAS), (dict(lse=dense((T, HQ), 0)), ALIAS),
    (dict(lse=dense((T, HQ), 20 * MB)), ALIAS), (dict(lse=dense((T, HQ), 2 * MB - 16)), ALIAS),
    (dict(out=view((T, HQ, 128), MB, (136, 128, 1))), ALIAS),                                       # heads of neighbouring tokens overlap
    (dict(ws=None), WORKSPACE), (dict(ws=BASE + 64 * MB + 16), WORKSPACE), (dict(nbytes=128), WORKSPACE),
]


@pytest.mark.parametrize("over,want", ATTN)
def test_attention_refusals(lib, over, want):  # noqa: F811
    assert attn(lib, **over) == want
    assert lib.kda_last_error()


def test_attention_workspace_size(lib):  # noqa: F811
    for bad in ((-1, 8, 2, 1, 1), (1, 0, 1, 1, 1), (1, 8, 0, 1, 1), (1, 8, 3, 1, 1), (1, 8, 2, -1, 1), (1, 8, 2, 1, -1), (1, 8, 2, 1, 1 << 40)):
        assert kb.kda_attn_qcache_workspace_size(*bad) == 0
    assert kb.kda_attn_qcache_workspace_size(0, 8, 2, 0, 0) >= 256
    need = kb.kda_attn_qcache_workspace_size(T, HQ, HK, N, S)
    assert attn(lib, nbytes=need - 1) == WORKSPACE


# ------------------------------------------------------------------ gated norm
def gated(lib, **over):
    a = dict(x=view((T, HK, 128), 0), gate=view((T, HK, 128), MB), w=dense((128,), 2 * MB), out=view((T, HK, 128), 3 * MB), eps=1e-6, flags=0)
    a.update(over)
    return lib.kda_gated_norm(a["x"], a["gate"], a["w"], a["out"], a["eps"], a["flags"], None)


GATED = [
    (dict(flags=2), INVALID), (dict(eps=NAN), INVALID), (dict(eps=-1.0), INVALID), (dict(x=None), INVALID), (dict(gate=None), INVALID), (dict(out=None), INVALID),
    (dict(x=view((T, HK, 64), 0)), UNSUPPORTED), (dict(x=view((T, HK, 128), 0, dtype=F32)), INVALID), (dict(gate=view((T, HK + 1, 128), MB)), INVALID),
    (dict(gate=view((T, HK, 128), MB + 8)), INVALID), (dict(out=view((T, HK, 128), 3 * MB, (0, 128, 1))), INVALID), (dict(w=dense((64,), 2 * MB)), INVALID),
    (dict(w=dense((128,), 2 * MB, BF)), INVALID), (dict(out=view((T, HK, 128), 256)), ALIAS), (dict(out=view((T, HK, 128), MB + 256)), ALIAS),
    (dict(out=view((T, HK, 128), 2 * MB)), ALIAS), (dict(x=view((T, 65536, 128), 0)), UNSUPPORTED),
    (dict(out=view((T, HK, 128), 3 * MB, (128, 128, 1))), ALIAS),
]


@pytest.mark.parametrize("over,want", GATED)
def test_gated_norm_refusals(lib, over, want):  # noqa: F811
    assert gated(lib, **over) == want
    assert lib.kda_last_error()


# ------------------------------------------------------------------ residual norm
DIM = 256


def residual(lib, **over):
    a = dict(y=view((T, DIM), 0), res=view((T, DIM), MB, dtype=F32), post=dense((DIM,), 2 * MB), gate=view((T, DIM), 3 * MB), scale=1.0, pre=dense((DIM,), 4 * MB),
             ro=view((T, DIM), 5 * MB, dtype=F32), out=view((T, DIM), 6 * MB), eps=1e-6)
    a.update(over)
    return lib.kda_residual_norm(a["y"], a["res"], a["post"], a["gate"], a["scale"], a["pre"], a["ro"], a["out"], a["eps"], None)


ALONE = dict(y=None, post=None, gate=None, ro=None)
RESIDUAL = [
    (dict(scale=NAN), INVALID), (dict(scale=float("inf")), INVALID), (dict(eps=NAN), INVALID), (dict(eps=-1e-9), INVALID), (dict(res=None), INVALID), (dict(out=None), INVALID),
    (dict(y=None), INVALID), (dict(ALONE, post=dense((DIM,), 2 * MB)), INVALID), (dict(ALONE, gate=view((T, DIM), 3 * MB)), INVALID),
    (dict(ALONE, ro=view((T, DIM), 5 * MB, dtype=F32)), INVALID), (dict(res=view((T, DIM), MB, dtype=I64)), INVALID), (dict(res=view((DIM,), MB, dtype=F32)), INVALID),
    (dict(y=view((T, DIM), 0, dtype=F32)), INVALID), (dict(y=view((T, DIM + 8), 0)), INVALID), (dict(y=view((T, DIM), 8)), INVALID), (dict(y=view((T, DIM), 0, (DIM, 2))), INVALID),
    (dict(y=view((T, DIM), 0, (DIM + 4, 1))), INVALID), (dict(y=view((T, DIM), 0, (DIM - 8, 1))), INVALID), (dict(y=view((T, DIM), 0, (0, 1))), INVALID),
    (dict(res=view((T, DIM), MB, (0, 1), F32)), INVALID), (dict(out=view((T, DIM), 6 * MB, (0, 1))), INVALID), (dict(ro=view((T, DIM), 5 * MB)), INVALID),
    (dict(gate=view((T, DIM), 3 * MB, (8, 1))), INVALID), (dict(post=dense((DIM + 8,), 2 * MB)), INVALID), (dict(pre=dense((DIM,), 4 * MB, BF)), INVALID),
    (dict(ALONE, res=view((T, 12), MB, dtype=F32), out=view((T, 12), 6 * MB), pre=None), UNSUPPORTED),
    (dict(ALONE, res=view((T, 16392), MB, dtype=F32), out=view((T, 16392), 8 * MB), pre=None), UNSUPPORTED),
    (dict(out=view((T, DIM), MB)), ALIAS), (dict(out=view((T, DIM), 5 * MB)), ALIAS), (dict(out=view((T, DIM), 3 * MB)), ALIAS), (dict(out=view((T, DIM), 2 * MB)), ALIAS),
    (dict(out=view((T, DIM), 256)), ALIAS), (dict(ro=view((T, DIM), 0, dtype=F32)), ALIAS), (dict(ro=view((T, DIM), MB + 64, dtype=F32)), ALIAS),
    (dict(ro=view((T, DIM), 4 * MB, dtype=F32)), ALIAS), (dict(gate=view((T, DIM), 6 * MB + 512, (0, 1))), ALIAS),
    (dict(res=view((T, DIM), MB), ro=view((T, DIM), 5 * MB), out=view((T, DIM), MB)), ALIAS),       # out over the stream, which is stored elsewhere
    (dict(res=view((T, DIM), MB), ro=view((T, DIM), MB), out=view((T, DIM), MB)), ALIAS),
]


@pytest.mark.parametrize("over,want", RESIDUAL)
def test_residual_norm_refusals(lib, over, want):  # noqa: F811
    assert residual(lib, **over) == want
    assert lib.kda_last_error()


# ------------------------------------------------------------------ the binding
@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(kb, "_lib", Library())


def calls(kind, space, status):
    bf, lens = tensors(kind, (4, 2, D))[0], tensors(kind, (1,), dtype=torch.int64)[0]
    c, row = tensors(kind, (1, 8, 2, ROW), dtype=torch.uint8)[0], tensors(kind, (4, 256))[0]
    return {
        "append": lambda: kb.kda_qcache_append(bf, bf, c, lens, status=status, stream=0),
        "attn": lambda: kb.kda_attn_qcache_fwd(bf, c, 1.0, bf, lens, workspace=space, stream=0),
        "gated": lambda: kb.kda_gated_norm(bf, bf, None, bf, stream=0),
        "residual": lambda: kb.kda_residual_norm(row, row, None, row, stream=0),
    }


@pytest.mark.parametrize("name", ["append", "attn", "gated", "residual"])
def test_devices(name, two_devices):
    with pytest.raises(ValueError, match="current device"):
        calls(On1, ws(On1), ws(On1))[name]()
    with pytest.raises(AssertionError, match="was called"):
        calls(On0, ws(On0), ws(On0))[name]()
    if name in ("append", "attn"):
        for other in (ws(On1), "no tensor"):
            with pytest.raises(ValueError, match="other tensors' device"):
                calls(On0, other, other)[name]()


def test_caches_of_the_binding(two_devices):
    bf, lens = tensors(On0, (4, 2, D))[0], tensors(On0, (1,), dtype=torch.int64)[0]
    for bad in (tensors(On0, (1, 8, 2, ROW))[0], tensors(On0, (8, 2, ROW), dtype=torch.uint8)[0], tensors(On1, (1, 8, 2, ROW), dtype=torch.uint8)[0]):
        for call in (lambda: kb.kda_qcache_append(bf, bf, bad, lens, stream=0), lambda: kb.kda_attn_qcache_fwd(bf, bad, 1.0, bf, lens, stream=0)):
            with pytest.raises(ValueError, match="cache"):
                call()
    with pytest.raises(TypeError, match="cache"):
        kb.kda_attn_qcache_fwd(bf, None, 1.0, bf, lens, stream=0)


def test_binding_constants():
    from test_abi_host import _header_constants
    consts = _header_constants()
    for name in ("KDA_U8", "KDA_QCACHE_ROW", "KDA_FLAG_GATE_SILU", "KDA_RESIDUAL_MAX_DIM"):
        assert getattr(kb, name) == consts[name]


@pytest.mark.parametrize("tokens,hq,hk,n,room", [(4096, 64, 8, 256, 131072), (20000, 64, 8, 32767, 4096), (300, 16, 8, 2, 1 << 27), (1 << 20, 8, 1, 32767, 1 << 30)])
def test_attention_workspace_is_bounded(lib, tokens, hq, hk, n, room):  # noqa: F811
    """4 GB of expanded keys and values, or one sequence's one head where that is more, besides the queries."""
    one = (-(-room // 128)) * (128 * (2 * 128 + 16) * 2 + 128 + 16)
    need = kb.kda_attn_qcache_workspace_size(tokens, hq, hk, n, room)
    assert 0 < need <= max(1 << 32, one) + tokens * hq * 292 + (64 << 20)


def test_attention_workspace_of_ordinary_caches(lib):  # noqa: F811
    """As many key heads of all sequences as fit into 1 GB; one of all of them up to 4 GB."""
    for n, room, hk, heads in ((4, 16384, 8, 8), (64, 4096, 8, 7), (64, 32768, 8, 1), (64, 100000, 8, 1)):
        unit = (room + 127) // 128 * (128 * (2 * 128 + 16) * 2 + 128 + 16)
        need = kb.kda_attn_qcache_workspace_size(1024 * n, 4 * hk, hk, n, room)
        keys = need - 1024 * n * 4 * heads * 292
        assert unit * n * heads <= keys <= unit * n * heads + (64 << 20)
