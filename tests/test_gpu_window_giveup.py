"""How the windowed attention kernels leave when a wait runs out in the middle
of their rings: in a test build with a short poll limit, one copy is left out
or comes late.  The call returns and says PA_DEVERR_TIMEOUT, the CTA starts
nothing more and leaves with nothing on its way, other requests and heads are
as without the fault, and the next call is clean."""

import json
import subprocess
import sys

import pytest

from tests.test_gpu_window_timeout import ROOT, test_lib  # noqa: F401  (test_lib: the fixture)

pytestmark = pytest.mark.gpu


def child(lib, name):
    r = subprocess.run([sys.executable, "-m", f"tests.{name}", lib], cwd=ROOT, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_decode_leaves_nothing_on_its_way(test_lib):  # noqa: F811
    records = child(test_lib, "window_giveup_child")
    assert len(records) == 6 * (1 + 16)
    for rec in records:
        if rec["box"] is None:
            assert rec["status"] == [0, 0, 0, 0] and rec["left"] == [0, 0], rec
            continue
        assert rec["status"][:3] == [0, 0, 0] and rec["status"][3] == 4, rec
        assert rec["left"] == [0, 0], rec
        # Request 0, kv head 0: four query heads.
        assert rec["rows"] and all(r == 0 and h < 4 for r, h in rec["rows"]), rec
        assert rec["after"] == [0, 0, 0, 0] and rec["left_after"] == [0, 0] and rec["same"], rec


def test_prefill_leaves_nothing_on_its_way(test_lib):  # noqa: F811
    for rec in child(test_lib, "window_giveup_prefill_child"):
        assert rec["plain"] == [0, 0, 0, 0] and rec["plain_left"] == 0, rec
        assert rec["muted"] == [0, 0, 0, 4] and rec["left"] == 0, rec
        # The muted unit, and those that the CTA had taken over by then.
        assert [0, 0] in rec["units"] and len(rec["units"]) <= 4, rec
        assert rec["after"] == [0, 0, 0, 0] and rec["left_after"] == 0 and rec["same"], rec
