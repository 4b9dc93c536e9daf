"""The bounded waits of the windowed attention kernels, made to run out: a
test build with a short poll limit and hooks under which one copy is never
issued.  The call returns, the error word says PA_DEVERR_TIMEOUT, the rows of
units that the failed CTA did not take are as without the fault, and the next
call is clean."""

import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def test_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_50_gb300 import build
    return build.build(extra_flags=["-DPA_TEST_HOOKS", "-DPA_WAIT_POLLS=4096"],
                       out_dir=os.path.join(build.PKG, "_build", "timeout_variant"),
                       lib_name="libpa_timeout.so")


def test_missing_copies_time_out_and_the_device_recovers(test_lib):
    r = subprocess.run([sys.executable, "-m", "tests.window_timeout_child", test_lib], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    rec = json.loads(r.stdout.strip().splitlines()[-1])
    for name in ("prefill", "decode"):
        got = rec[name]
        assert got["plain"] == [0, 0, 0], (name, got)
        assert got["skipped"][:2] == [0, 0] and got["skipped"][2] & 4, (name, got)
        assert [0, 0] in got["differ"], (name, got)
        assert len(got["differ"]) <= (3 if name == "prefill" else 1), (name, got)
        assert got["after"] == [0, 0, 0] and got["same"], (name, got)
