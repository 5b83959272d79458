"""Which tensors of the mixers' C ABI may share memory (no GPU; the addresses are fake and never
dereferenced): a written tensor that meets a read one is refused, one whose elements only lie between the
other's is not.  A call that passes all of those checks stops at the workspace, which is missing here."""
import random

import pytest

from gated_delta_rule_36_gb300 import binding as kb
from test_mixers_host import ALIAS, BF, I64, INVALID, MB, WORKSPACE, dense, lib, lin, rope, step, view  # noqa: F401

T, H, D = 6, 3, 128
STATE, STATE2 = (1, H, D, D), (2, H, D, D)


@pytest.mark.parametrize("over", [
    dict(final=dense(STATE, 3 * MB - 4096)),                                            # log_decay lies in it
    dict(final=dense(STATE, 8 * MB), cu=dense((2,), 8 * MB + 64, I64)),                 # so do the lengths
    dict(final=dense(STATE, 8 * MB, BF), cu=dense((2,), 8 * MB + 3 * D * D * 2 - 16, I64)),
], ids=["log_decay", "cu_seqlens", "cu_seqlens_end"])
def test_lin_fwd_final_state_over_what_is_read(lib, over):  # noqa: F811
    assert lin(lib, **over) == ALIAS
    assert b"final_state" in lib.kda_last_error()


def test_lin_fwd_final_state_beside_the_lengths(lib):  # noqa: F811
    assert lin(lib, final=dense(STATE, 8 * MB, BF), cu=dense((2,), 8 * MB + 3 * D * D * 2, I64), ws=0) == WORKSPACE


def test_lin_decode_final_state_over_log_decay(lib):  # noqa: F811
    assert step(lib, final=dense(STATE2, 3 * MB - 4096)) == ALIAS
    assert b"final_state" in lib.kda_last_error()


def strides_of(shape):
    s, n = [], 1
    for x in reversed(shape):
        s.insert(0, n)
        n *= x
    return s


def part(shape, keep, index, batch=None):
    """The view of a buffer of `shape` at 0 that keeps the dimensions `keep` (token, head, 128) and fixes the
    others at `index` (a dictionary); with a batch dimension in front."""
    st = strides_of(shape)
    at = sum(2 * st[d] * i for d, i in index.items())
    dims = [shape[d] for d in keep]
    stride = [st[d] for d in keep]
    if batch is None:
        return view((1, *dims), at, (dims[0] * stride[0], *stride))
    return view((batch, dims[0] // batch, *dims[1:]), at, (dims[0] // batch * stride[0], *stride))


BUFFERS = {   # q, k, v and out side by side in one buffer: columns of a projection, heads in turn, planes
    "columns": ((T, 4, H, D), (0, 2, 3), 1), "heads_in_turn": ((T, H, 4, D), (0, 1, 3), 2), "planes": ((4, T, H, D), (1, 2, 3), 0),
    "heads_outside": ((H, T, 4, D), (1, 0, 3), 2), "heads_outside_planes": ((H, 4, T, D), (2, 0, 3), 1), "wide": ((T, H, 4, 2 * D), None, None),
}


@pytest.mark.parametrize("batch", [None, 2])
@pytest.mark.parametrize("name", BUFFERS)
def test_parts_of_one_buffer_that_do_not_meet(lib, name, batch):  # noqa: F811
    shape, keep, fixed = BUFFERS[name]
    if keep is None:      # rows of 256 of which each tensor has a half
        at = lambda i: 2 * D * (i & 1) + 4 * D * (i >> 1)
        one = lambda i: view((1, T, H, D), at(i), (T * H * 8 * D, H * 8 * D, 8 * D, 1))
        views = [one(i) for i in range(4)]
    else:
        views = [part(shape, keep, {fixed: i}, batch) for i in range(4)]
    q, k, v, out = views
    assert lin(lib, q=q, k=k, v=v, out=out, ld=dense((H,), 3 * MB), ws=0) == WORKSPACE, lib.kda_last_error()


@pytest.mark.parametrize("shift", [-248, -128, -8, 0, 8, 120, 248, 512, 512 * (H * T - 1) + 248])
def test_parts_of_one_buffer_that_meet(lib, shift):  # noqa: F811
    """Heads in turn, of 512 elements each: q has elements 0 to 255 (as two heads), out as many from `shift` on."""
    of = lambda at: view((1, T * H, 2, D), at, (T * H * 4 * D, 4 * D, D, 1))
    far = dict(k=view((1, T * H, 2, D), 8 * MB), v=view((1, T * H, 2, D), 9 * MB), ld=dense((2,), 10 * MB), ws=0)
    assert lin(lib, q=of(MB), out=of(MB + 2 * shift), **far) == ALIAS
    for apart in (256, -256, 512 * T * H):
        assert lin(lib, q=of(MB), out=of(MB + 2 * apart), **far) == WORKSPACE


def test_any_two_views_that_share_an_element_are_refused(lib):  # noqa: F811
    """Drawn views of small strides against a set of their elements."""
    r = random.Random(1)
    refused = passed = 0
    for _ in range(3000):
        h, t = r.choice([1, 2, 3]), r.choice([1, 2, 5])

        def drawn(at):
            st = [D * r.choice([1, 2, 3, 4, 6, 8, 12, 24]) + r.choice([0, 0, 8]) for _ in range(2)]
            return at, st, view((1, t, h, D), 2 * at, (10 ** 6, *st, 1))

        def elements(at, st):
            return {at + i * st[0] + j * st[1] + d for i in range(t) for j in range(h) for d in range(0, D, 8)}

        (a0, sa, va), (b0, sb, vb) = drawn(8 * r.randint(0, 400)), drawn(8 * r.randint(0, 400))
        meet = bool(elements(a0, sa) & elements(b0, sb))
        far = dict(k=view((1, t, h, D), 8 * MB), v=view((1, t, h, D), 9 * MB), ld=dense((h,), 10 * MB), ws=0)
        got = lin(lib, q=va, out=vb, **far)
        assert got in (ALIAS, WORKSPACE)
        assert got == ALIAS or not meet, (a0, sa, b0, sb, t, h)
        refused += got == ALIAS and not meet
        passed += not meet
    assert refused < 0.4 * passed      # (strides that do not nest may be refused without need)


def test_sizes_that_fit_no_memory(lib):  # noqa: F811
    st = (1 << 37, 1 << 37, D, 1)
    far = dict(k=view((1, 1 << 20, H, D), 8 * MB, st), v=view((1, 1 << 20, H, D), 9 * MB, st), out=view((1, 1 << 20, H, D), 4 * MB, st))
    assert lin(lib, q=view((1, 1 << 20, H, D), 0, st), ws=0, **far) == INVALID
    assert rope(lib, cs=dense((1 << 60, 64), 4 * MB)) == INVALID
