"""The bounded waits of the attention over a 4-bit cache run out, on the GPU, in the form that faults nothing: in a child
process with the test-only build (tests/wait_qcache.py), which has a time limit.
"""
import os
import subprocess
import sys

import pytest

from gated_delta_rule_36_gb300 import build as kbuild

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_expired_waits_return_the_timeout_status():
    env = dict(os.environ, KDA_LIBRARY=kbuild.build(variant="waittest"))
    env.pop("KDA_TEST_SKIP_SHARE", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/wait_qcache.py"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
