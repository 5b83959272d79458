"""The residual norm where a block takes several rows, one after another, in every type and width of the stream."""
import pytest
import torch

import gated_delta_rule_36_gb300 as kda
from test_gpu_mixers import gen_of, rand, within
from test_gpu_norms import nan, ref_residual

pytestmark = pytest.mark.gpu


# at least 16 blocks an SM hold rows at once: so many tokens are several rows for each (four for the rows of a warp)
@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,T", [(128, 40001), (256, 20003), (264, 8001), (1024, 7001), (2304, 5003), (4096, 5001), (4104, 4001), (8192, 3001), (8200, 3001), (16384, 1501)])
def test_residual_norm_of_many_tokens(dim, T, dtype, gate):
    g = gen_of(dim)
    y, res = rand(g, T, dim), rand(g, T, dim, dtype=dtype)
    gt = None if gate is None else rand(g, T, dim) if gate == "token" else rand(g, 1, dim).expand(T, dim)
    w, pw = rand(g, dim, dtype=torch.float32), rand(g, dim, dtype=torch.float32)
    for post in (pw, None):
        out, ro = nan(T, dim), nan(T, dim, dtype=dtype)
        r, rb, o, ob = ref_residual(y, res, post, gt, 0.5, w, 1e-6)
        kda.kda_residual_norm(y, res, w, out, residual_out=ro, post_weight=post, gate=gt, scale=0.5)
        within("residual_out", ro, r, rb)
        within("out", out, o, ob)
        del r, rb, o, ob
    y2, res2 = y.clone(), res.clone()                                    # in place: the next row is loaded before this one is written
    kda.kda_residual_norm(y2, res2, w, y2, residual_out=res2, gate=gt, scale=0.5)
    assert torch.equal(y2, out) and torch.equal(res2, ro)
    alone = nan(T, dim)
    kda.kda_residual_norm(None, res, w, alone)
    _, _, o, ob = ref_residual(None, res, None, None, 1.0, w, 1e-6)
    within("norm alone", alone, o, ob)
