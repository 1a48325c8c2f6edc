"""ffd_decode_tree's waits run out, without a GPU fault.

The debug build takes a limit for them (none, or a few microseconds, no more than a
tile takes to come).  The call must end, with all of a CTA's waits at once, report
FFD_DEVICE_FLAG_TIMEOUT, write nothing outside its output and workspace, and with the
usual limit give the result that it gave before (debug_tree_wait_run.py, in a process
of its own: a process loads one of the two libraries)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_short_limits_end_the_call_and_are_reported():
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_tree_wait_run.py")],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "ended and were reported" in r.stdout
