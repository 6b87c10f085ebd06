"""Calls of the shared-prefix, scored and evicting operators that the host answers by itself: sizes, refusals, and where the
binding's own memory comes from.  No GPU."""
import os
import subprocess
import sys

import pytest

from tests.test_operators_cpu import A, B_, Cc, D_, INVALID, P, WORKSPACE, coded, evict, message, scored, shared

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


# what a call writes and what it reads: A, B_, Cc, D_ lie far apart, and arrays of the small shapes end well before the next
FAR = 0x90000000


@pytest.mark.parametrize("call", [shared, coded, scored])
@pytest.mark.parametrize("kw,word", [
    (dict(out=P(A + 64)), "q"), (dict(lse=P(A + 64)), "q"), (dict(lse=P(Cc + 16)), "out"), (dict(lse=P(B_ + 4)), "lens"),
    (dict(starts=P(Cc + 8)), "starts"), (dict(oo=P(FAR), ol=P(Cc)), "other_lse"), (dict(oo=P(FAR), ol=P(A), lse=P(FAR + 4)), "other_out"),
    (dict(ws=P(Cc + 16)), "workspace"), (dict(ws=P(A)), "workspace")])
def test_attention_refuses_outputs_over_other_arrays(call, kw, word):
    kw = dict(kw) if call is scored else dict(kw, rows=200)
    assert call(**kw) == INVALID
    assert "overlaps" in message() and word in message()


@pytest.mark.parametrize("kw,word", [
    (dict(so=P(A + 32)), "q"), (dict(so=P(Cc)), "score_out"), (dict(so=P(FAR + 4), oo=P(FAR), ol=P(A)), "other_out"),
    (dict(so=P(D_ + 64)), "workspace"), (dict(lse=P(0x50000000 + 4)), "lse")])
def test_scored_refuses_scores_over_other_arrays(kw, word):
    assert scored(**kw) == INVALID
    assert "overlaps" in message() and word in message()


@pytest.mark.parametrize("kw,word", [
    (dict(lo=P(0x70001000)), "next_pos"), (dict(lo=P(0x70001000), nx=P(0x70001000)), "next_pos"), (dict(lo=P(0x70001004)), "next_pos"),
    (dict(so=P(0x60000000)), "pos"), (dict(po=P(0x50000000)), "score"), (dict(so=P(FAR), po=P(FAR + 16)), "score_out"),
    (dict(lo=P(0x50000010)), "score"), (dict(ws=P(0x60000000)), "workspace"), (dict(ws=P(0x70001000)), "workspace")])
def test_evict_refuses_outputs_over_other_arrays(kw, word):
    """lens_out = next_pos above all: a head's CTA wrote the length while others of the sequence still read the position."""
    assert evict(**kw) == INVALID
    assert "overlaps" in message() and word in message()
    assert evict(**dict(kw, max_len=-1)) == INVALID and "max_len" in message()


def test_evict_takes_one_array_of_lengths_and_positions():
    """Nothing evicted yet: the next position is the length.  In place the call is sound (refused here for its workspace only)."""
    one = P(0x70000000)
    assert evict(li=one, nx=one, lo=one, ws=None) == WORKSPACE
    assert evict(li=one, nx=one, lo=P(0x70000004), ws=None) == WORKSPACE
    assert evict(li=one, nx=one, lo=P(0x70000004)) == INVALID
