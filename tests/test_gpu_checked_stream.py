"""The calls for long streams in a paged cache under the bounds-checked build (see
test_gpu_checked.py): page-table entries, queries, boxes and slots, decoded tiles, output rows and
copied pages are held against their extents.  Parity runs in a child process on that library; no
check may fail."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.environ.get("QPS_LIB_VARIANT") == "checked"


@pytest.mark.skipif(CHECKED, reason="the parent run starts the checked child run")
def test_stream_calls_pass_under_the_checked_build():
    from quantized_position_split_gb300 import build
    build.build(variant="checked")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_prompt.py",
           "tests/test_gpu_window.py", "tests/test_gpu_pages.py", "tests/test_gpu_checked_stream.py",
           "-k", "not many_tiles and not never_comes and not multi_query and not large_pool"]
    res = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, QPS_LIB_VARIANT="checked"), capture_output=True, text=True,
                         timeout=1200)
    tail = (res.stdout + res.stderr)[-4000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "failed" not in res.stdout, tail


@pytest.mark.skipif(not CHECKED, reason="runs in the checked child process")
def test_no_check_failed():
    """(last in the child run)"""
    import quantized_position_split_gb300 as qps
    assert qps.lib().qps_build_checked() == 1
    qps.device_status(reset=True)
