"""Calls of the shared-prefix, scored and evicting operators that the host answers by itself: sizes, refusals, and where the
binding's own memory comes from.  No GPU."""
import os
import subprocess
import sys

import pytest
import torch

import looped_lm_decode_b200 as LQ
import looped_lm_decode_b200.loopvq as binding
from tests.test_operators_cpu import A, B_, Cc, D_, INVALID, P, UNSUPPORTED, WORKSPACE, coded, desc, evict, message, scored, shared

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


def test_scored_refuses_more_rows_than_its_maps_hold():
    """2^31 rows of keys are 275 GB at 64 channels."""
    d = desc(B=64, Hkv=1 << 10, Hq=1 << 12, D=64, Nmax=1 << 15)
    assert scored(d, max_len=64) == UNSUPPORTED and "2^31" in message()


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


# ------------------------------------------------------------------ the binding's own memory

class OnHost:
    """The binding's calls with host tensors: the GPU check passes and the launch is a stub that takes what the library's
    checks would take (a cache at an odd address, or of a code width that is not built, is refused)."""

    def __init__(self, monkeypatch):
        self.sizes = []
        real = LQ.lib()

        class Lib:
            def __getattr__(_, name):
                fn = getattr(real, name)
                if name in ("loopvq_bf16_shared_attn", "loopvq_shared_attn", "loopvq_bf16_decode_attn_scored", "loopvq_bf16_evict"):
                    def call(desc, *args):
                        self.sizes.append(args[-2])
                        x = desc._obj
                        return 1 if (getattr(x, "k", 0) or 0) % 16 or getattr(x, "c", 4) not in (4, 8, 16, 32) else 0
                    return call
                return fn

        monkeypatch.setattr(binding, "lib", lambda: Lib())
        monkeypatch.setattr(binding, "_need_current", lambda device, stream: device)
        monkeypatch.setattr(binding, "_stream", lambda stream: None)
        monkeypatch.setattr(binding, "_on_stream", lambda *_: None)
        monkeypatch.setattr(binding, "_sizes", {})


def aligned(n, off=0):
    """n bf16 elements at an address that is a multiple of 16, or two bytes behind one."""
    x = torch.empty(n + 16, dtype=torch.bfloat16)                    # (never read; filling it would start threads)
    at = (-x.data_ptr() // 2) % 8 + off
    return x[at:at + n]


def odd_and_right(hkv, n, d, hq):
    make = lambda off: LQ.Bf16Cache(aligned(hkv * n * d, off).view(1, hkv, n, d), aligned(hkv * n * d).view(1, hkv, n, d), hq)  # noqa: E731
    return make(1), make(0)


@pytest.mark.parametrize("op", ["shared", "scored", "evict"])
def test_a_refused_cache_leaves_no_size_behind(monkeypatch, op):
    """The library answers a size of 0 for a cache that it refuses; a right call of the same shape gets its own."""
    host = OnHost(monkeypatch)
    odd, right = odd_and_right(2, 32768, 64, 2)
    q, lens, score = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.empty(1, 2, 32768)
    pos = torch.empty(1, 2, 32768, dtype=torch.int32)
    call = dict(shared=lambda c: LQ.bf16_shared_attn(c, 0, q, lens, 32768),
                scored=lambda c: LQ.bf16_decode_attn_scored(c, q, lens, 32768, score),
                evict=lambda c: LQ.bf16_evict(c, score, pos, lens, lens, 32768, 100, 4, 8))[op]
    with pytest.raises(LQ.LoopVQError):
        call(odd)
    call(right)
    call(right)                                                      # from what was kept
    want = dict(shared=LQ.bf16_shared_workspace_bytes(right, 1, 32768), scored=LQ.bf16_scored_workspace_bytes(right, 32768),
                evict=LQ.bf16_evict_workspace_bytes(right, 32768, 100))[op]
    assert want > 0 and host.sizes == [0, want, want]


def test_a_refused_coded_cache_leaves_no_size_behind(monkeypatch):
    host = OnHost(monkeypatch)
    q, lens = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)

    def cache(c):
        x = LQ.Cache(1, 4, 4, 2, 2, 64, c, 256, 1, 32768, alloc=False)
        x.idx = x.codebook = x.slices = x.rope = torch.zeros(16)
        return x

    with pytest.raises(LQ.LoopVQError):
        LQ.shared_attn(cache(6), 0, 0, 0, q, lens, 32768)
    LQ.shared_attn(cache(4), 0, 0, 0, q, lens, 32768)
    want = LQ.shared_workspace_bytes(cache(4), 3, 32768)
    assert want > 0 and host.sizes == [0, want]


@pytest.mark.parametrize("stream", [None, "side"])
def test_own_memory_is_made_on_the_stream_that_uses_it(monkeypatch, stream):
    """Results and workspaces that the caller leaves to the binding."""
    OnHost(monkeypatch)
    current, made = [None], []

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *_):
            current.pop()

    real = torch.empty_strided
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch, "empty_strided", lambda *a, **k: (made.append(current[-1]), real(*a, **k))[1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *_: None)
    _, cache = odd_and_right(2, 32768, 64, 2)
    q, lens, score = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.empty(1, 2, 32768)
    pos = torch.empty(1, 2, 32768, dtype=torch.int32)
    coded = LQ.Cache(1, 4, 4, 2, 2, 64, 4, 256, 1, 32768, alloc=False)
    coded.idx = coded.codebook = coded.slices = coded.rope = torch.zeros(16)
    LQ.bf16_shared_attn(cache, 0, q, lens, 32768, stream=stream)
    LQ.shared_attn(coded, 0, 0, 0, q, lens, 32768, stream=stream)
    LQ.bf16_decode_attn_scored(cache, q, lens, 32768, score, stream=stream)
    LQ.bf16_evict(cache, score, pos, lens, lens, 32768, 100, 4, 8, stream=stream)
    assert made == [stream] * 10                                     # three results and workspaces, and evict's workspace


@pytest.mark.parametrize("stream", [None, "side"])
def test_own_memory_of_every_decode_call(monkeypatch, stream):
    """decode_attn and its kin, merge2 and dequant_debug: the launch is a stub, what they make comes from the right stream,
    and results are recorded for the current one."""
    made, results = [], []
    monkeypatch.setattr(binding, "_empty", lambda shape, strides, dtype, device, s: (
        made.append(s), torch.empty_strided(shape, strides, dtype=dtype, device="cpu"))[1])
    monkeypatch.setattr(binding, "_new_like", lambda t, s: (made.append(s), torch.empty_like(t))[1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: "here")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: results.append(s))
    monkeypatch.setattr(binding, "_stream", lambda s: None)
    real = LQ.lib()

    class Lib:
        def __getattr__(_, name):
            return getattr(real, name) if name.endswith("_bytes") or name.endswith("_elems") else lambda *a: 0

    monkeypatch.setattr(binding, "lib", lambda: Lib())
    cache = LQ.Cache(1, 4, 4, 2, 2, 64, 4, 256, 1, 512, alloc=False)
    bf = LQ.Bf16Cache(aligned(2 * 512 * 64).view(1, 2, 512, 64), aligned(2 * 512 * 64).view(1, 2, 512, 64), 2)
    tasq, win = LQ.Tasq(cache, device="cpu"), LQ.Window(cache, 8, 8, device="cpu")
    q, lens = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    kv, part = torch.zeros(1, 2, 64, dtype=torch.bfloat16), (torch.zeros(1, 2, 64), torch.zeros(1, 2))
    on = dict(stream=stream)
    LQ.decode_attn(cache, 0, 0, q, lens, 512, **on)
    LQ.decode_attn_noalloc(cache, 0, 0, q, lens, 512, **on)
    LQ.decode_attn_range(cache, 0, 0, q, None, lens, 512, **on)
    LQ.bf16_decode_attn(bf, q, lens, 512, **on)
    LQ.tasq_decode_attn(cache, tasq, 0, 0, q, lens, 512, **on)
    LQ.window_decode_attn(win, cache, 0, 0, q, 512, **on)
    LQ.window_append_decode_attn(win, cache, 0, 0, kv, kv, kv, q, 512, **on)
    LQ.merge2(*part, *part, **on)
    LQ.dequant_debug(cache, 0, 0, 0, 0, 0, 8, **on)
    assert made == [stream] * (6 * 3 + 2 + 2 + 1)
    assert results == (["here"] * (6 * 2 + 2 + 1) if stream else [])
