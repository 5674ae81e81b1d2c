"""The 4-bit KV cache's GPU tests once more against the bounds-checked library (every raw
global access checked against its tensor's extent; see test_gpu_bounds_checked.py)."""
import os
import subprocess
import sys

import pytest

from differential_attention_05_b200 import build as B

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_kv4_under_the_bounds_checked_library():
    assert os.path.exists(B.LIB_DEBUG), "libdiffattn_debug.so is missing: python -m differential_attention_05_b200.build --debug"
    env = dict(os.environ, DIFFATTN_LIBRARY=B.LIB_DEBUG, DIFFATTN_EXPECT_NO_VIOLATIONS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           os.path.join(HERE, "test_gpu_kv4.py")]
    r = subprocess.run(cmd, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert "0 out-of-range accesses skipped" in r.stdout, tail


def test_kv4_accuracy_and_calls_under_the_bounds_checked_library():
    env = dict(os.environ, DIFFATTN_LIBRARY=B.LIB_DEBUG, DIFFATTN_EXPECT_NO_VIOLATIONS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           *(os.path.join(HERE, f"test_gpu_kv4_{name}.py") for name in ("branches", "scales", "calls"))]
    r = subprocess.run(cmd, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert "0 out-of-range accesses skipped" in r.stdout, tail
