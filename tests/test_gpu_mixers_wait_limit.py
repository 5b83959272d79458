"""A mixer's wait for another share's state in memory has the limit of its other waits, and no share's report is
lost: in child processes with the test-only build (tests/wait_limit_mixers.py, tests/wait_status_mixers.py), which have
a time limit.
"""
import os
import subprocess
import sys

import pytest

from gated_delta_rule_36_gb300 import build as kbuild

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tests", ["wait_limit_mixers.py", "wait_status_mixers.py"])
def test_with_the_test_only_build(tests):
    env = dict(os.environ, KDA_LIBRARY=kbuild.build(variant="waittest"))
    env.pop("KDA_TEST_SKIP_SHARE", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-m", "gpu", "-p", "no:cacheprovider",
                        f"tests/{tests}"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
