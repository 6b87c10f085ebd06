"""Calls of the shared-prefix, scored and evicting operators that the host answers by itself: sizes, refusals, and where the
binding's own memory comes from.  No GPU."""
import os
import subprocess
import sys

from tests.test_operators_cpu import INVALID, coded, message, shared

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_workspace_of_no_rows():
    """A batch may be empty: no rows need no workspace (asked in a process of its own, which a signal would end)."""
    code = ("import ctypes as C, looped_lm_decode_b200 as LQ; from tests.test_operators_cpu import desc, coded_desc; L = LQ.lib()\n"
            "for n in (0, 1, 700, 4096):\n"
            "    assert L.loopvq_bf16_shared_workspace_bytes(C.byref(desc()), 0, n) == 0\n"
            "    assert L.loopvq_shared_workspace_bytes(C.byref(coded_desc()), 0, n) == 0\n")
    assert subprocess.run([sys.executable, "-c", code], timeout=300, cwd=ROOT).returncode == 0


def test_no_rows_are_checked_like_any():
    for call in (shared, coded):
        assert call(rows=0, seq=2) == INVALID and "seq" in message()
