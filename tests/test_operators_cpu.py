"""Refusals of the shared-prefix, scored and evicting calls, and their workspace sizes: checked on the host before any
launch, so they need no GPU."""
import ctypes as C
import math

import pytest
import torch

import looped_lm_decode_b200 as LQ

P = lambda x: C.c_void_p(x)  # noqa: E731
A, B_, Cc, D_ = 0x10000000, 0x20000000, 0x30000000, 0x40000000       # far apart, 16-byte aligned, never read
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def desc(B=2, Hkv=2, Hq=4, D=128, Nmax=4096, k=A, v=B_):
    return LQ.Bf16CacheDesc(B, Hkv, Hq, D, Nmax, k, v)


def coded_desc(**kw):
    f = dict(L=1, T=4, Tc=4, Hkv=2, Hq=2, D=128, c=4, K=256, B=2, Nmax=4096, theta=1e4, idx=A, codebook=B_, slices=Cc,
             rope=D_, ncb=1)
    f.update(kw)
    return LQ.CacheDesc(*[f[n] for n, _ in LQ.CacheDesc._fields_])


def message():
    return LQ.lib().loopvq_last_error().decode()


def shared(d=None, **kw):
    f = dict(seq=0, q=P(A), rows=3, starts=None, lens=P(B_), max_len=4096, scale=0.0, oo=None, ol=None, out=P(Cc), lse=None,
             ws=P(D_), n=1 << 40)
    f.update(kw)
    return LQ.lib().loopvq_bf16_shared_attn(C.byref(d or desc()), f["seq"], f["q"], f["rows"], f["starts"], f["lens"],
                                            f["max_len"], f["scale"], f["oo"], f["ol"], f["out"], f["lse"], f["ws"],
                                            f["n"], None)


def coded(d=None, layer=0, t=0, **kw):
    f = dict(seq=0, q=P(A), rows=3, starts=None, lens=P(B_), max_len=4096, scale=0.0, oo=None, ol=None, out=P(Cc), lse=None,
             ws=P(D_), n=1 << 40)
    f.update(kw)
    return LQ.lib().loopvq_shared_attn(C.byref(d or coded_desc()), layer, t, f["seq"], f["q"], f["rows"], f["starts"],
                                       f["lens"], f["max_len"], f["scale"], f["oo"], f["ol"], f["out"], f["lse"],
                                       f["ws"], f["n"], None)


BAD = [
    (dict(seq=-1), INVALID, "seq"), (dict(seq=2), INVALID, "seq"), (dict(rows=-1), INVALID, "rows"),
    (dict(q=None), INVALID, "q"), (dict(q=P(A + 2)), INVALID, "aligned"), (dict(lens=None), INVALID, "lens"),
    (dict(lens=P(B_ + 1)), INVALID, "lens"), (dict(starts=P(B_ + 2)), INVALID, "starts"), (dict(out=None), INVALID, "out"),
    (dict(lse=P(D_ + 2)), INVALID, "lse"), (dict(max_len=-1), INVALID, "max_len"), (dict(max_len=4097), INVALID, "max_len"),
    (dict(scale=math.nan), INVALID, "scale"), (dict(scale=math.inf), INVALID, "scale"),
    (dict(oo=P(A)), INVALID, "together"), (dict(ol=P(A)), INVALID, "together"),
    (dict(oo=P(Cc + 16), ol=P(A)), INVALID, "overlaps"), (dict(oo=P(A), ol=P(D_), lse=P(D_)), INVALID, "lse"),
    (dict(oo=P(A), ol=P(D_), lse=P(D_ + 4)), INVALID, "lse"),
    (dict(ws=None), WORKSPACE, "workspace"), (dict(n=100), WORKSPACE, "workspace"), (dict(ws=P(D_ + 8)), INVALID, "workspace"),
    (dict(rows=1 << 30), UNSUPPORTED, "large"),
]


@pytest.mark.parametrize("kw,status,word", BAD)
@pytest.mark.parametrize("call", [shared, coded])
def test_shared_refuses(call, kw, status, word):
    assert call(**kw) == status
    assert word in message()


def test_shared_refuses_shapes():
    for kw, status in ((dict(D=96), UNSUPPORTED), (dict(Hq=6), UNSUPPORTED), (dict(Hq=5), INVALID), (dict(k=None), INVALID),
                       (dict(v=B_ + 2), INVALID), (dict(Hkv=1 << 15, Hq=1 << 15, Nmax=1 << 17), UNSUPPORTED)):
        assert shared(desc(**kw), max_len=64) == status, kw
    for kw, status in ((dict(c=6), UNSUPPORTED), (dict(idx=None), INVALID), (dict(slices=None), INVALID),
                       (dict(rope=D_ + 4), INVALID), (dict(ncb=7), INVALID)):
        assert coded(coded_desc(**kw)) == status, kw
    assert coded(layer=1) == INVALID and coded(layer=-1) == INVALID and coded(t=4) == INVALID and coded(t=-1) == INVALID


def test_no_rows_launch_nothing():
    assert shared(rows=0, q=None, lens=None, out=None, ws=None, n=0) == 0
    assert coded(rows=0, q=None, lens=None, out=None, ws=None, n=0) == 0


def scored(d=None, **kw):
    f = dict(q=P(A), starts=None, lens=P(B_), max_len=4096, scale=0.0, oo=None, ol=None, si=None, so=P(0x50000000), out=P(Cc),
             lse=None, ws=P(D_), n=1 << 40)
    f.update(kw)
    return LQ.lib().loopvq_bf16_decode_attn_scored(C.byref(d or desc()), f["q"], f["starts"], f["lens"], f["max_len"],
                                                   f["scale"], f["oo"], f["ol"], f["si"], f["so"], f["out"], f["lse"],
                                                   f["ws"], f["n"], None)


@pytest.mark.parametrize("kw,status,word", [b for b in BAD if not {"seq", "rows"} & set(b[0])] + [
    (dict(so=None), INVALID, "score_out"), (dict(so=P(0x50000002)), INVALID, "score_out"),
    (dict(si=P(0x50000000 + 64)), INVALID, "overlaps"), (dict(si=P(0x50000001)), INVALID, "score_in")])
def test_scored_refuses(kw, status, word):
    assert scored(**kw) == status
    assert word in message()


def evict(d=None, **kw):
    f = dict(si=P(0x50000000), pi=P(0x60000000), li=P(0x70000000), nx=P(0x70001000), max_len=4096, budget=1024, sink=8,
             recent=64, so=P(0x50000000), po=P(0x60000000), lo=P(0x70000000), ws=P(D_), n=1 << 40)
    f.update(kw)
    return LQ.lib().loopvq_bf16_evict(C.byref(d or desc()), f["si"], f["pi"], f["li"], f["nx"], f["max_len"], f["budget"],
                                      f["sink"], f["recent"], f["so"], f["po"], f["lo"], f["ws"], f["n"], None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(budget=0), INVALID, "budget"), (dict(budget=-5), INVALID, "budget"), (dict(sink=-1), INVALID, "n_sink"),
    (dict(recent=-1), INVALID, "n_recent"), (dict(sink=1000, recent=25), INVALID, "budget"),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID, "budget"), (dict(max_len=4097), INVALID, "max_len"),
    (dict(max_len=-1), INVALID, "max_len"), (dict(si=None), INVALID, "score_in"), (dict(pi=None), INVALID, "pos_in"),
    (dict(li=None), INVALID, "lens_in"), (dict(nx=None), INVALID, "next_pos"), (dict(so=None), INVALID, "score_out"),
    (dict(po=P(0x60000002)), INVALID, "pos_out"), (dict(lo=None), INVALID, "lens_out"),
    (dict(so=P(0x50000004)), INVALID, "score_out"), (dict(po=P(0x60000004)), INVALID, "pos_out"),
    (dict(lo=P(0x70000004)), INVALID, "lens_out"), (dict(ws=None), WORKSPACE, "workspace"),
    (dict(n=64), WORKSPACE, "workspace"), (dict(ws=P(D_ + 4)), INVALID, "workspace")])
def test_evict_refuses(kw, status, word):
    assert evict(**kw) == status
    assert word in message()


def test_evict_refuses_too_many_heads():
    assert evict(desc(B=70000, Hkv=1, Hq=1, Nmax=4), max_len=4, budget=100) == UNSUPPORTED


def test_workspace_sizes():
    L, d = LQ.lib(), desc()
    big, coded_d = desc(Nmax=32768), coded_desc(Nmax=32768)
    assert L.loopvq_bf16_shared_workspace_bytes(C.byref(big), 3, 32768) > 0
    assert L.loopvq_shared_workspace_bytes(C.byref(coded_d), 3, 32768) > 0
    assert L.loopvq_bf16_shared_workspace_bytes(C.byref(d), 3, 5000) == 0            # past Nmax
    assert L.loopvq_bf16_shared_workspace_bytes(C.byref(d), 3, 500) == 0             # one launch, none needed
    assert L.loopvq_bf16_evict_workspace_bytes(C.byref(d), 2049, 2048) == 0
    assert L.loopvq_bf16_evict_workspace_bytes(C.byref(d), 4096, 1024) >= 4 * 4 * (1 + 2 * 1024)
    assert L.loopvq_bf16_evict_workspace_bytes(C.byref(d), 4096, 0) == 0
    # more rows and longer prefixes never need less
    sizes = [L.loopvq_bf16_shared_workspace_bytes(C.byref(big), r, 32768) for r in (1, 4, 16, 33, 64, 65, 300)]
    assert all(s > 0 for s in sizes)
    assert L.loopvq_bf16_shared_workspace_bytes(C.byref(big), 2 ** 31 - 1, 32768) == 0   # more rows than a call takes
    assert shared(big, rows=2 ** 31 - 1, max_len=32768) == UNSUPPORTED
    # a batch's scores alone: 4 bytes a token and query head
    assert L.loopvq_bf16_scored_workspace_bytes(C.byref(desc(B=64, Hkv=4, Hq=16)), 4096) >= 64 * 16 * 4096 * 4


def test_python_refuses_host_memory():
    k = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    cache = LQ.Bf16Cache(k, k.clone(), 2)
    q, lens, score = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64)
    for call in (lambda: LQ.bf16_shared_attn(cache, 0, q, lens, 64),
                 lambda: LQ.bf16_decode_attn_scored(cache, q, lens, 64, score),
                 lambda: LQ.bf16_evict(cache, score, score.int(), lens, lens, 64, 32, 4, 8)):
        with pytest.raises(LQ.LoopVQError) as e:
            call()
        assert e.value.status == INVALID and "GPU" in str(e.value)
