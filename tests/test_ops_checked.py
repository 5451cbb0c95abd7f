"""The operators around the layer on the bounds-checked build: their own tests again in a child
pytest (KDA_TEST_CHECKED=1, see conftest.py), where every device-error read also fails if a
kernel recorded an index outside its buffer."""
import os
import subprocess
import sys

import pytest

from gated_delta_rule_48_gb300 import binding as kb

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_on_the_checked_build():
    if os.environ.get("KDA_TEST_CHECKED") == "1":
        pytest.skip("already the checked run")
    kb.build(checked=True)
    env = dict(os.environ, KDA_TEST_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
                        "tests/test_norm.py", "tests/test_matmul_fp8.py", "tests/test_short_conv.py",
                        "tests/test_ssm_scan.py", "tests/test_example_block.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
