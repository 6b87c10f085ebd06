"""Attention of many query tokens over one sequence (a shared prefix), bf16 and coded, against plain fp64 forms.

Tolerances.  Scores: products of bf16 values are exact, a tensor-core sum of D of them in fp32 is taken as off by at most
8 roundings of 2^-22 of sum |q k| scale, which for normal inputs is about 0.64 sqrt(D) < 8: 2e-5.  Two bf16 parts hold a
value to 2^-17 of itself (the first is off by 2^-8 of its binade at most, the second by 2^-9 of what is left): a rebuilt
key, rotated in fp32 (4 roundings, angles of the fp32 table: 2^-22), gives 8 (2^-17 + 2^-22) = 6.3e-5, P (held in two or
three parts) 7.6e-6.  A weight is then off by at most DELTA = 1e-4 of itself; sums over tokens add up to some hundred
accumulations of 2^-23, 4e-5.  An output is held to 2 DELTA + 4e-5 < 2.5e-4 of sum p |v|, a log-sum-exp to DELTA."""
import math

import pytest
import torch

import looped_lm_decode_b200 as LQ

pytestmark = pytest.mark.gpu

DELTA = 1e-4
OUT = 2.5e-4


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reference(q, k, v, other, scale=None):
    """q [R][Hq][D], k and v [Hkv][n][D] in fp64: out, lse and sum p |v| of the joint softmax."""
    R, Hq, D = q.shape
    Hkv, n = k.shape[:2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    x = q.double().view(R, Hkv, Hq // Hkv, D)
    s = torch.einsum("rhgd,hnd->rhgn", x, k) * scale
    lse = torch.logsumexp(s, 3) if n else torch.full(s.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    joint = lse if other is None else torch.logaddexp(lse, other[1].double().view(R, Hkv, -1))
    at = torch.where(joint == -math.inf, 0.0, joint)
    p = torch.exp(s - at[..., None])
    out, mag = torch.einsum("rhgn,hnd->rhgd", p, v), torch.einsum("rhgn,hnd->rhgd", p, v.abs())
    if other is not None:
        po = torch.exp(other[1].double().view(R, Hkv, -1) - at)[..., None]
        oo = other[0].double().view(R, Hkv, -1, D)
        out, mag = out + po * oo, mag + po * oo.abs()
    return out.reshape(R, Hq, D), joint.reshape(R, Hq), mag.reshape(R, Hq, D)


def check(got, ref):
    out, lse = got
    ro, rl, mag = ref
    err = (out.double() - ro).abs()
    assert (err <= OUT * mag).all(), f"{(err / (mag + 1e-30)).max().item():.3g} of sum p |v|"
    empty = rl == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    assert ((lse.double() - rl)[~empty].abs() <= DELTA).all()


def make_other(g, rows, hq, d):
    other = (torch.randn(rows, hq, d, generator=g, device="cuda"),
             3 + 3 * torch.randn(rows, hq, generator=g, device="cuda"))
    other[0][0, 0], other[1][0, 0] = 0, -math.inf
    return other


def run_bf16(n, rows, hkv, hq, d, start=0, seqs=1, seq=0, pad=5, scale=0.0, seed=0):
    g = gen(seed + n * 31 + rows)
    cache = LQ.Bf16Cache(bf16(g, seqs, hkv, n + pad, d), bf16(g, seqs, hkv, n + pad, d), hq)
    q = bf16(g, rows, hq, d)
    k, v = (x[seq, :, start:n].double() for x in (cache.k, cache.v))
    lens, starts = i32([n if i == seq else 1 for i in range(seqs)]), i32([start if i == seq else 0 for i in range(seqs)])
    for other in (None, make_other(g, rows, hq, d)):
        got = LQ.bf16_shared_attn(cache, seq, q, lens, n, starts=starts if start else None, other=other, scale=scale)
        LQ.fault_check()
        check(got, reference(q, k, v, other, scale or None))


@pytest.mark.parametrize("n", [1, 2, 15, 64, 127, 128, 129, 256, 1000])
@pytest.mark.parametrize("rows", [1, 3, 127, 128, 129])
def test_bf16_lengths_and_rows(n, rows):
    run_bf16(n, rows, 2, 2, 128)


@pytest.mark.parametrize("hkv,hq,d", [(1, 1, 64), (3, 6, 64), (2, 8, 128), (4, 32, 128), (1, 8, 64), (5, 5, 128)])
@pytest.mark.parametrize("n,rows", [(77, 5), (700, 33), (5003, 70)])
def test_bf16_heads(hkv, hq, d, n, rows):
    run_bf16(n, rows, hkv, hq, d)


@pytest.mark.parametrize("n,start,seqs,seq", [(300, 1, 1, 0), (300, 130, 2, 1), (300, 299, 3, 2), (1025, 511, 2, 0)])
def test_bf16_ranges_and_sequences(n, start, seqs, seq):
    run_bf16(n, 9, 2, 4, 128, start, seqs, seq, pad=3)
    run_bf16(n, 150, 2, 2, 64, start, seqs, seq, pad=0)


@pytest.mark.parametrize("rows", [600, 2000])
def test_bf16_many_rows(rows):
    run_bf16(2111, rows, 1, 2, 128)


@pytest.mark.parametrize("n", [0, 1, 100, 257, 385, 513, 1024, 1025])
@pytest.mark.parametrize("rows,hkv,hq", [(33, 1, 1), (140, 2, 2), (70, 16, 32), (600, 40, 40)])
def test_results_with_and_without_records(rows, hkv, hq, n):
    """One launch that writes the result, or records and a merge: every side of the rules that choose, into the other part's
    own memory, with empty parts."""
    g = gen(13 + n)
    cache = LQ.Bf16Cache(bf16(g, 1, hkv, max(n, 8), 64), bf16(g, 1, hkv, max(n, 8), 64), hq)
    q, lens = bf16(g, rows, hq, 64), i32([n])
    other = make_other(g, rows, hq, 64)
    other[1][:, -1] = -math.inf
    want = reference(q, cache.k[0, :, :n].double(), cache.v[0, :, :n].double(), (torch.where(
        other[1][..., None] == -math.inf, 0.0, other[0]), other[1]))
    out = other[0].clone()
    got = LQ.bf16_shared_attn(cache, 0, q, lens, n, other=(out, other[1]), out=out)
    LQ.fault_check()
    assert got[0].data_ptr() == out.data_ptr()
    check(got, want)


def test_bf16_long_and_scaled():
    run_bf16(40001, 4, 1, 1, 128)
    run_bf16(3001, 20, 2, 2, 128, scale=0.01)
    run_bf16(3001, 20, 2, 2, 64, scale=0.5)


def test_bf16_rising_scores():
    """Scores that grow along the tokens move the running maximum tile after tile."""
    g = gen(3)
    n, rows, d = 2000, 140, 128
    cache = LQ.Bf16Cache(bf16(g, 1, 1, n, d), bf16(g, 1, 1, n, d), 1)
    q = bf16(g, rows, 1, d)
    q[:, :, 0] = 8
    cache.k[:, :, :, 0] = torch.linspace(-60, 60, n, device="cuda").bfloat16()
    ref = reference(q, cache.k[0].double(), cache.v[0].double(), None)
    out, lse = LQ.bf16_shared_attn(cache, 0, q, i32([n]), n)
    # |q k| reaches 480 / sqrt(D): the score's share of the tolerance grows with it
    grow = 1 + 8 * 60 / math.sqrt(d) / 8
    assert ((out.double() - ref[0]).abs() <= OUT * grow * ref[2]).all()
    assert ((lse.double() - ref[1]).abs() <= DELTA * grow).all()


def test_bf16_empty_and_clamped():
    g = gen(4)
    cache = LQ.Bf16Cache(bf16(g, 2, 2, 64, 128), bf16(g, 2, 2, 64, 128), 2)
    q = bf16(g, 3, 2, 128)
    other = make_other(g, 3, 2, 128)
    for lens, starts, max_len in (([0, 9], None, 64), ([9, 9], [9, 0], 64), ([9, 9], None, 0), ([-4, 9], [-3, 1], 64)):
        s = None if starts is None else i32(starts)
        out, lse = LQ.bf16_shared_attn(cache, 0, q, i32(lens), max_len, starts=s)
        assert (out == 0).all() and (lse == -math.inf).all()
        out, lse = LQ.bf16_shared_attn(cache, 0, q, i32(lens), max_len, starts=s, other=other)
        assert torch.equal(out, other[0]) and torch.allclose(lse, other[1], rtol=1e-6, atol=0)
    out, lse = LQ.bf16_shared_attn(cache, 1, q, i32([0, 1000]), 50)
    check((out, lse), reference(q, cache.k[1, :, :50].double(), cache.v[1, :, :50].double(), None))
    out, lse = LQ.bf16_shared_attn(cache, 1, q[:0], i32([0, 1000]), 50)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)


@pytest.mark.parametrize("rows", [5, 200])
def test_bf16_masked_values_are_not_seen(rows):
    """Infinities and NaN before the start, behind the length and in the other sequences change nothing."""
    g = gen(5)
    cache = LQ.Bf16Cache(bf16(g, 3, 2, 400, 128), bf16(g, 3, 2, 400, 128), 2)
    q = bf16(g, rows, 2, 128)
    args = (cache, 1, q, i32([400, 301, 400]), 400)
    clean = LQ.bf16_shared_attn(*args, starts=i32([0, 37, 0]))
    for x in (cache.k, cache.v):
        x[0], x[2] = math.nan, math.inf
        x[1, :, :37], x[1, :, 301:] = math.inf, math.nan
    dirty = LQ.bf16_shared_attn(*args, starts=i32([0, 37, 0]))
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("rows", [5, 25, 100, 300])
@pytest.mark.parametrize("n", [300, 3000])
def test_nan_stays_in_its_row_and_is_not_lost(rows, n):
    """A query or another part of NaN makes its row NaN, with tokens or without, and no other row differs."""
    g = gen(11)
    cache = LQ.Bf16Cache(bf16(g, 2, 2, n, 128), bf16(g, 2, 2, n, 128), 2)
    coded = make_coded(g, 2, 2, 128, 4, 4, 1, 256, 2, n)
    q, lens = bf16(g, rows, 2, 128), i32([n, 0])
    other = make_other(g, rows, 2, 128)
    bad_q, bad_o = q.clone(), (other[0], other[1].clone())
    bad_q[3, 1, 5] = math.nan
    bad_o[1][2, 0] = math.nan
    hit = torch.zeros(rows, 2, dtype=torch.bool, device="cuda")
    for call in (lambda x, o, s: LQ.bf16_shared_attn(cache, s, x, lens, n, other=o),
                 lambda x, o, s: LQ.shared_attn(coded, 0, 1, s, x, lens, n, other=o)):
        for x, o, s, at in ((bad_q, None, 0, (3, 1)), (q, bad_o, 0, (2, 0)), (q, bad_o, 1, (2, 0))):
            good, bad = call(q, None if o is None else other, s), call(x, o, s)
            hit[:] = False
            hit[at] = True
            assert bad[0][hit].isnan().all() and bad[1][hit].isnan().all()
            assert torch.equal(good[0][~hit], bad[0][~hit]) and torch.equal(good[1][~hit], bad[1][~hit])


# ------------------------------------------------------------------ coded

def make_coded(g, hkv, hq, d, c, tc, ncb, entries, seqs, nmax, loops=4):
    cache = LQ.Cache(1, loops, tc, hkv, hq, d, c, entries, seqs, nmax, ncb=ncb)
    cache.codebook.copy_(bf16(g, cache.codebook.numel()).view(torch.int16))
    LQ.prepare(cache)
    code = torch.randint(0, entries, (cache.idx.numel(), 4), generator=g, device="cuda")
    words = (code * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], device="cuda")).sum(1)
    cache.idx.copy_(torch.where(words >= 2 ** 31, words - 2 ** 32, words).int())
    return cache


def rebuild(cache, t, seq, start, n):
    """Keys (rotated) and values [Hkv][n - start][D] in fp64, from words, codebooks and fp64 angles."""
    c, d, tc, hkv, ncb = cache.c, cache.D, cache.Tc, cache.Hkv, cache.ncb
    groups, np_ = d // c, d // (2 * c)
    block, m = divmod(t, tc)
    words = cache.idx.view(cache.L, cache.NB, cache.B, hkv, cache.Nmax // 4, np_, 4)[0, block, seq].long() % 2 ** 32
    tok = torch.arange(start, n, device="cuda")
    books = cache.codebook.view(torch.bfloat16).view(cache.L, cache.NB, 2, hkv, ncb, cache.K, c * tc)[0, block].double()
    head = torch.arange(hkv, device="cuda")[:, None]
    out = []
    for kv in range(2):
        x = torch.zeros(hkv, n - start, d, dtype=torch.float64, device="cuda")
        for grp in range(groups):
            w = words[:, tok // 4, grp % np_, tok % 4]
            code = (w >> (8 * (2 * kv + grp // np_))) & 255
            x[:, :, grp * c:(grp + 1) * c] = books[kv, head, grp if ncb > 1 else 0, code][:, :, m::tc]
        out.append(x)
    k, h = out[0], d // 2
    ang = tok.double()[:, None] * cache.theta ** (-2.0 * torch.arange(h, dtype=torch.float64, device="cuda") / d)
    cos, sin = torch.cos(ang), torch.sin(ang)
    return torch.cat([k[..., :h] * cos - k[..., h:] * sin, k[..., h:] * cos + k[..., :h] * sin], -1), out[1]


def run_coded(n, rows, hkv, hq, d, c, tc, ncb=1, entries=256, start=0, seqs=1, seq=0, t=1):
    g = gen(n * 17 + rows + c)
    cache = make_coded(g, hkv, hq, d, c, tc, ncb, entries, seqs, (n + 3) // 4 * 4)
    q = bf16(g, rows, hq, d)
    k, v = rebuild(cache, t, seq, start, n)
    lens, starts = i32([n if i == seq else 1 for i in range(seqs)]), i32([start if i == seq else 0 for i in range(seqs)])
    for other in (None, make_other(g, rows, hq, d)):
        got = LQ.shared_attn(cache, 0, t, seq, q, lens, n, starts=starts if start else None, other=other)
        LQ.fault_check()
        check(got, reference(q, k, v, other))


@pytest.mark.parametrize("n", [1, 3, 63, 64, 65, 128, 1001])
@pytest.mark.parametrize("rows", [1, 100, 130])
def test_coded_lengths_and_rows(n, rows):
    run_coded(n, rows, 2, 2, 128, 4, 4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c,tc", [(4, 4), (4, 1), (8, 4), (8, 2), (16, 2), (16, 1), (32, 1)])
@pytest.mark.parametrize("per_group", [False, True])
@pytest.mark.parametrize("rows", [6, 70])
def test_coded_shapes(d, c, tc, per_group, rows):
    for t in range(4):
        run_coded(333, rows, 2, 4, d, c, tc, d // c if per_group else 1, t=t)


@pytest.mark.parametrize("hkv,hq,d", [(1, 1, 64), (3, 3, 128), (2, 16, 128), (1, 8, 64)])
@pytest.mark.parametrize("n,start,seqs,seq", [(500, 0, 1, 0), (500, 1, 2, 1), (501, 66, 3, 0), (777, 776, 1, 0)])
def test_coded_heads_ranges_and_sequences(hkv, hq, d, n, start, seqs, seq):
    run_coded(n, 11, hkv, hq, d, 4, 4, start=start, seqs=seqs, seq=seq, t=3)
    run_coded(n, 90, hkv, hq, d, 8, 4, start=start, seqs=seqs, seq=seq, entries=100, t=2)


def test_coded_long():
    run_coded(30001, 20, 2, 2, 128, 4, 4)
    run_coded(9999, 140, 1, 1, 64, 4, 4, entries=7)


def test_coded_empty_and_garbage_behind_the_length():
    g = gen(6)
    cache = make_coded(g, 2, 2, 128, 4, 4, 1, 256, 2, 400)
    q = bf16(g, 4, 2, 128)
    out, lse = LQ.shared_attn(cache, 0, 0, 1, q, i32([4, 0]), 400)
    assert (out == 0).all() and (lse == -math.inf).all()
    args = (cache, 0, 2, 1, q, i32([0, 201]), 400)
    clean = LQ.shared_attn(*args, starts=i32([0, 7]))
    words = cache.idx.view(2, 2, 100, -1, 4)
    words[0] = -1
    words[1, :, :1] = -1                                             # tokens 0 .. 3, before the start
    words[1, :, 51:] = 12345                                         # tokens 204 .., behind the length
    dirty = LQ.shared_attn(*args, starts=i32([0, 7]))
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


# ------------------------------------------------------------------ in use

def test_prefix_then_own_tokens_then_eviction():
    """A decode step of a batch behind a shared prefix: the prefix part joins the scored decode over each sequence's
    own cache, whose weights are those of the joint softmax; then the caches evict.  Both orders of merging agree."""
    b, hkv, hq, d, n_prefix, n_own = 6, 2, 8, 128, 900, 300
    g = gen(7)
    q = bf16(g, b, hq, d)
    own = LQ.Bf16Cache(bf16(g, b, hkv, n_own, d), bf16(g, b, hkv, n_own, d), hq)
    lens = i32([300, 1, 0, 128, 77, 299])
    prefix = LQ.Bf16Cache(bf16(g, 1, hkv, n_prefix, d), bf16(g, 1, hkv, n_prefix, d), hq)
    coded = make_coded(g, hkv, hq, d, 8, 4, 1, 256, 1, n_prefix)
    k, v = prefix.k[0].double(), prefix.v[0].double()
    kc, vc = rebuild(coded, 1, 0, 0, n_prefix)
    calls = ((lambda **kw: LQ.bf16_shared_attn(prefix, 0, q, i32([n_prefix]), n_prefix, **kw), k, v),
             (lambda **kw: LQ.shared_attn(coded, 0, 1, 0, q, i32([n_prefix]), n_prefix, **kw), kc, vc))
    for shared, kk, vv in calls:
        part = shared()
        score = torch.zeros(b, hkv, n_own, device="cuda")
        out, lse, score = LQ.bf16_decode_attn_scored(own, q, lens, n_own, score, other=part)
        first = LQ.bf16_decode_attn(own, q, lens, n_own)
        out2, lse2 = shared(other=first)
        into = (first[0].clone(), first[1].clone())
        out3, lse3 = shared(other=into, out=into[0])                 # in place
        assert torch.equal(out2, out3) and torch.equal(lse2, lse3)
        for i in range(b):
            n = int(lens[i])
            ki, vi = torch.cat([kk, own.k[i, :, :n].double()], 1), torch.cat([vv, own.v[i, :, :n].double()], 1)
            ref = reference(q[i:i + 1], ki, vi, None)
            check((out[i:i + 1], lse[i:i + 1]), ref)
            check((out2[i:i + 1], lse2[i:i + 1]), ref)
            s = torch.einsum("hgd,hnd->hgn", q[i].double().view(hkv, -1, d), own.k[i, :, :n].double()) / math.sqrt(d)
            w = torch.exp(s - ref[1].view(hkv, -1, 1)).sum(1)
            assert ((score[i, :, :n] - w).abs() <= 2 * DELTA * w).all() and (score[i, :, n:] == 0).all()
        pos = (n_prefix + torch.arange(n_own, device="cuda", dtype=torch.int32)).expand(b, hkv, n_own).contiguous()
        after = lens.clone()
        LQ.bf16_evict(own, score, pos, after, lens + n_prefix, n_own, 100, n_sink=0, n_recent=32)
        assert after.tolist() == [100, 1, 0, 100, 77, 100]
        out, lse = LQ.bf16_decode_attn(own, q, after, n_own)
        assert out.isfinite().all()
        lens = after.clone()


@pytest.mark.parametrize("rows", [4, 200])
def test_repeated_captured_and_on_other_streams(rows):
    g = gen(8)
    n, hkv, hq, d = 1500, 2, 2, 128
    cache = LQ.Bf16Cache(bf16(g, 1, hkv, n, d), bf16(g, 1, hkv, n, d), hq)
    coded = make_coded(g, hkv, hq, d, 4, 4, 1, 256, 1, n)
    q, lens = bf16(g, rows, hq, d), i32([n])
    eager = LQ.bf16_shared_attn(cache, 0, q, lens, n), LQ.shared_attn(coded, 0, 1, 0, q, lens, n)
    for _ in range(20):                                              # equal inputs give equal bits
        again = LQ.bf16_shared_attn(cache, 0, q, lens, n), LQ.shared_attn(coded, 0, 1, 0, q, lens, n)
        for x, y in zip(eager, again):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    outs = [torch.empty_like(eager[0][0]) for _ in range(4)]
    lses = [torch.empty_like(eager[0][1]) for _ in range(4)]
    ws = [torch.empty(LQ.bf16_shared_workspace_bytes(cache, rows, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    wc = [torch.empty(LQ.shared_workspace_bytes(coded, rows, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        LQ.bf16_shared_attn(cache, 0, q, lens, n, out=outs[0], lse=lses[0], workspace=ws[0])
        LQ.shared_attn(coded, 0, 1, 0, q, lens, n, out=outs[1], lse=lses[1], workspace=wc[0])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], eager[i][0]) and torch.equal(lses[i], eager[i][1])
    # two calls at once, on two streams
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        LQ.bf16_shared_attn(cache, 0, q, lens, n, out=outs[2], lse=lses[2], workspace=ws[1], stream=a)
        LQ.shared_attn(coded, 0, 1, 0, q, lens, n, out=outs[3], lse=lses[3], workspace=wc[1], stream=b)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[2 + i], eager[i][0]) and torch.equal(lses[2 + i], eager[i][1])


@pytest.mark.parametrize("rows,n", [(4, 700), (200, 700), (200, 252), (90, 252)])
def test_a_wait_that_runs_out_is_reported(rows, n):
    """With a limit of 0 every wait tests once and gives up: NaN rows, a fault, and the next call works."""
    g = gen(9)
    cache = LQ.Bf16Cache(bf16(g, 1, 1, n, 128), bf16(g, 1, 1, n, 128), 1)
    coded = make_coded(g, 1, 1, 128, 4, 4, 1, 256, 1, n)
    q, lens = bf16(g, rows, 1, 128), i32([n])
    calls = (lambda: LQ.bf16_shared_attn(cache, 0, q, lens, n), lambda: LQ.shared_attn(coded, 0, 1, 0, q, lens, n))
    for call in calls:
        good = call()
        LQ.fault_check()
        before = LQ.wait_limit_ns()
        LQ.set_wait_limit_ns(0)
        try:
            bad = call()
            with pytest.raises(LQ.LoopVQError) as e:
                LQ.fault_check()
            assert e.value.status == 5 and "shared-prefix" in str(e.value)
            assert bad[0].isnan().all() and bad[1].isnan().all()
        finally:
            LQ.set_wait_limit_ns(before)
        after = call()
        LQ.fault_check()
        assert torch.equal(good[0], after[0]) and torch.equal(good[1], after[1])


def test_python_refuses_what_the_kernels_would_misread():
    g = gen(10)
    cache = LQ.Bf16Cache(bf16(g, 2, 2, 64, 64), bf16(g, 2, 2, 64, 64), 4)
    q, lens, score = bf16(g, 2, 4, 64), i32([64, 9]), torch.zeros(2, 2, 64, device="cuda")
    pos, ok = torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda"), dict(max_len=64)
    other = (torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 4, device="cuda"))
    bad = [
        lambda: LQ.bf16_shared_attn(cache, 0, q.float(), lens, **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q[:, :2], lens, **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q.transpose(0, 1).contiguous().transpose(0, 1), lens, **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens.long(), **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens[:1], **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens.cpu(), **ok),
        lambda: LQ.bf16_shared_attn(cache, 2, q, lens, **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens, starts=lens[:1], **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens, other=(other[0][:1], other[1]), **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens, other=other, lse=other[1], **ok),
        lambda: LQ.bf16_shared_attn(cache, 0, q, lens, out=other[0].double(), **ok),
        lambda: LQ.bf16_decode_attn_scored(cache, q, lens, 64, None),
        lambda: LQ.bf16_decode_attn_scored(cache, q, lens, 64, score[:, :1]),
        lambda: LQ.bf16_decode_attn_scored(cache, q, lens, 65, score),
        lambda: LQ.bf16_evict(cache, score, pos.long(), lens, lens, 64, 32, 4, 8),
        lambda: LQ.bf16_evict(cache, score.half(), pos, lens, lens, 64, 32, 4, 8),
        lambda: LQ.bf16_evict(cache, score, pos, lens, lens, 64, 8, 4, 8),
    ]
    for call in bad:
        with pytest.raises(LQ.LoopVQError):
            call()
    torch.cuda.synchronize()
