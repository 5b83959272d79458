"""Which tensors of the mixers' C ABI may share memory (no GPU; the addresses are fake and never
dereferenced): a written tensor that meets a read one is refused, one whose elements only lie between the
other's is not.  A call that passes all of those checks stops at the workspace, which is missing here."""
import pytest

from gated_delta_rule_36_gb300 import binding as kb
from test_mixers_host import ALIAS, BF, F32, I64, MB, WORKSPACE, dense, lib, lin, step, view  # noqa: F401

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
