"""The norms around the mixers on the GPU, against their formulas in 64 bits.

Bounds, per element, with u the unit roundoff of the output's type (bf16 2^-8):
  gated       u |y| for the output's rounding, 2^-17 |y| for the fp32 arithmetic (the gate's exponential included,
              whose argument of at most 16 log2(e) is rounded to 24 bits)
  residual    r: u |r| + 2^-18 (|residual| + |scale gate u|); out: u |out|, and those errors of the unrounded r
              (2^-18 of its terms) times the factor that turns r into out
"""
import math

import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import D, NAN, U, gen_of, rand, within

pytestmark = pytest.mark.gpu


def nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ gated norm
def ref_gated(x, gate, weight, eps, silu):
    x, a = x.double(), gate.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if weight is None else weight.double())
    y = y * a.sigmoid() * (a if silu else 1.0)
    return y, (U * 1.01 + 2.0 ** -17) * y.abs() + 1e-37


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T,h,fused,weighted", [
    (1, 1, False, True), (3, 5, True, True), (8, 32, True, False), (129, 7, False, True), (1000, 64, True, True), (2000, 33, False, False), (5, 96, True, True)])
def test_gated_norm(T, h, fused, weighted, silu):
    g = gen_of(T + h)
    x = rand(g, T, h, D, mul=3.0)
    gate = rand(g, T, 3 * h * D, mul=2.0)[:, h * D:2 * h * D].unflatten(1, (h, D)) if fused else rand(g, T, h, D, mul=2.0)
    x[T // 2] = 0.0
    w = rand(g, D, dtype=torch.float32) if weighted else None
    flags = kda.KDA_FLAG_GATE_SILU if silu else 0
    out = nan(T, h, D)
    kept = x.clone(), gate.clone()
    kda.kda_gated_norm(x, gate, w, out, flags=flags)
    ref, bound = ref_gated(x, gate, w, 1e-6, silu)
    within("out", out, ref, bound)
    assert torch.equal(x, kept[0]) and torch.equal(gate, kept[1])
    for which in range(2):                                               # in place of x, and of the gate
        a, b = kept[0].clone(), gate if which else kept[1]
        into = b if which else a
        kda.kda_gated_norm(a, b, w, into, flags=flags)
        assert torch.equal(into, out)


def test_gated_norm_of_extreme_gates_and_strides():
    g = gen_of(3)
    T, h = 9, 4
    buf = rand(g, h, T, 2 * D)
    x = buf[..., :D].transpose(0, 1)                                     # heads outside, gaps inside
    gate = torch.linspace(-16, 16, T * h * D, device="cuda").bfloat16().reshape(T, h, D)
    out = nan(h, T, 3 * D)
    view = out[..., D:2 * D].transpose(0, 1)
    kda.kda_gated_norm(x, gate, None, view, eps=1e-3)
    ref, bound = ref_gated(x, gate, None, 1e-3, False)
    within("out", view, ref, bound)
    assert torch.isnan(out[..., :D]).all() and torch.isnan(out[..., 2 * D:]).all()
    gate[0], gate[1], gate[2] = 300.0, -300.0, math.inf
    kda.kda_gated_norm(x, gate, None, view, eps=1e-3)
    ref, bound = ref_gated(x, gate, None, 1e-3, False)
    within("out", view, ref, bound + 2.0 ** -126)
    x[4, 1, 7] = math.inf
    kda.kda_gated_norm(x, gate, None, view)
    assert torch.isnan(view[4, 1, 7]) and (view[4, 1, 8:] == 0).all() and torch.isfinite(view[4, 0]).all()
    kda.kda_gated_norm(x[:0], gate[:0], None, view[:0])                  # no tokens


# ------------------------------------------------------------------ residual norm
def ref_residual(y, res, post, gate, scale, pre, eps):
    r = res.double()
    size = r.abs()
    if y is not None:
        u = y.double()
        if post is not None:
            u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * post.double()
        if gate is not None:
            u = u * gate.double()
        r, size = r + scale * u, size + (scale * u).abs()
    f = 1.0 / (r.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if pre is None else pre.double())
    out = r * f
    unit = U if res.dtype == torch.bfloat16 else 2.0 ** -24
    # the norm's own sum is off by as much of its terms: size * |size| summed is at most what the largest factor makes of it
    drift = 2.0 ** -18 * (size.square().mean(-1, keepdim=True) / (r.square().mean(-1, keepdim=True) + eps)).sqrt()
    return r, unit * 1.01 * r.abs() + 2.0 ** -18 * size, out, (U * 1.01 + 2.0 ** -18 + drift) * out.abs() + 2.0 ** -18 * size * f.abs() + 1e-37


DIMS = [8, 24, 128, 256, 264, 1000, 1024, 2048, 2304, 4096, 4104, 5120, 8192, 8200, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,gate,T", [(False, None, 5), (True, None, 33), (True, "token", 7), (False, "channel", 130), (True, "channel", 1)])
def test_residual_norm(dim, dtype, post, gate, T):
    g = gen_of(dim + T)
    y = rand(g, T, dim + 16, mul=3.0)[:, 8:8 + dim] if T > 1 else rand(g, T, dim)
    res = rand(g, T, dim, mul=2.0, dtype=dtype)
    y[T // 2] = 0.0
    pw, w = (rand(g, dim, dtype=torch.float32, mul=0.3) + 1.0 for _ in range(2))
    gt = None if gate is None else rand(g, T, dim) if gate == "token" else rand(g, 1, dim).expand(T, dim)
    kw = dict(post_weight=pw if post else None, gate=gt, scale=-0.375)
    ro, out = nan(T, dim + 8, dtype=dtype)[:, :dim], nan(T, dim)
    kept = y.clone(), res.clone()
    kda.kda_residual_norm(y, res, w, out, residual_out=ro, **kw)
    r, rb, o, ob = ref_residual(y, res, kw["post_weight"], gt, -0.375, w, 1e-6)
    within("residual_out", ro, r, rb)
    within("out", out, o, ob)
    assert torch.equal(y, kept[0]) and torch.equal(res, kept[1])
    # the stream and the block's output in place
    kda.kda_residual_norm(y, res, w, y, residual_out=res, **kw)
    assert torch.equal(res, ro) and torch.equal(y, out)
    # without the stream's output, and the norm alone
    again = nan(T, dim)
    kda.kda_residual_norm(kept[0], kept[1], w, again, **kw)
    assert torch.equal(again, out)
    kda.kda_residual_norm(None, kept[1], None, again, eps=1e-3)
    _, _, o, ob = ref_residual(None, kept[1], None, None, 1.0, None, 1e-3)
    within("norm alone", again, o, ob)
    if dtype == torch.bfloat16:
        alone = kept[1].clone()
        kda.kda_residual_norm(None, alone, None, alone, eps=1e-3)
        assert torch.equal(alone, again)


@pytest.mark.parametrize("dim,T", [(4096, 3000), (512, 20000), (2304, 1500), (5120, 900), (8192, 1100)])
def test_residual_norm_of_many_tokens(dim, T):
    g = gen_of(dim)
    y, res, gt = rand(g, T, dim), rand(g, T, dim, dtype=torch.float32), rand(g, T, dim)
    w, pw = rand(g, dim, dtype=torch.float32), rand(g, dim, dtype=torch.float32)
    out = nan(T, dim)
    r, rb, o, ob = ref_residual(y, res, pw, gt, 0.5, w, 1e-6)
    kda.kda_residual_norm(y, res, w, out, residual_out=res, post_weight=pw, gate=gt, scale=0.5)
    within("residual_out", res, r, rb)
    within("out", out, o, ob)


def test_residual_norm_of_zeros_nothing_and_bad_values():
    g = gen_of(4)
    z = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    out, ro = nan(3, 256), nan(3, 256)
    kda.kda_residual_norm(z, z, None, out, residual_out=ro, post_weight=torch.ones(256, device="cuda"))
    assert (out == 0).all() and (ro == 0).all()
    y = rand(g, 3, 256)
    y[1, 5] = NAN
    kda.kda_residual_norm(y, z, None, out, residual_out=ro)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()      # a token's norm is its own
    assert torch.isnan(ro[1, 5]) and torch.isfinite(ro[1, 6:]).all()
    kda.kda_residual_norm(y[:0], z[:0], None, out[:0])                           # no tokens
    graph = torch.cuda.CUDAGraph()
    y2, want = rand(g, 3, 256), nan(3, 256)
    with torch.cuda.graph(graph):
        kda.kda_residual_norm(y, z, None, out, residual_out=ro)
    y.copy_(y2)
    graph.replay()
    kda.kda_residual_norm(y2, z, None, want)
    assert torch.equal(out, want)


def test_captured_and_replayed_over_many_tokens():
    """More rows than one wave of blocks, in one graph, replayed on new inputs."""
    g = gen_of(5)
    T, dim, h = 3000, 1024, 40
    y, res, w = rand(g, T, dim), rand(g, T, dim, dtype=torch.float32), rand(g, dim, dtype=torch.float32)
    x, gate, out, out2 = rand(g, T, h, D), rand(g, T, h, D), nan(T, dim), nan(T, h, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_residual_norm(y, res, w, out, scale=0.5)
        kda.kda_gated_norm(x, gate, None, out2)
    for t in (y, res, x, gate):
        t.copy_(rand(g, *t.shape))
    graph.replay()
    want, want2 = nan(T, dim), nan(T, h, D)
    kda.kda_residual_norm(y, res, w, want, scale=0.5)
    kda.kda_gated_norm(x, gate, None, want2)
    assert torch.equal(out, want) and torch.equal(out2, want2)
    _, _, o, ob = ref_residual(y, res, None, None, 0.5, w, 1e-6)
    within("out", out, o, ob)
    ref, bound = ref_gated(x, gate, None, 1e-6, False)
    within("gated", out2, ref, bound)
