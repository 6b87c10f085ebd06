"""Scored decode attention and eviction on the GPU, against plain fp64 forms.

Tolerances, before any run.  A score is a sum of D products in fp32 (8 per lane in pairs, then 4 exchanges, the
query rounded once for the scale): under 24 roundings of relative size 2^-24 against sum |q k| scale, about
sqrt(D) for normal inputs, at most 2e-5; ex2 adds 2^-22, so a weight is off by at most DELTA = 4e-5 of itself with
the log-sum-exp's own error (a tensor-core sum of the exact products, 8 roundings of 2^-22, is within the same 2e-5).  Sums over tokens run in fp32 over at most some hundred terms per lane: 2^-24 each
against the sum of absolute terms.  An output is held to 2 DELTA + 1e-4 / 4 < 1.1e-4 of sum p |v|."""
import math

import pytest
import torch

import looped_lm_decode_b200 as LQ

pytestmark = pytest.mark.gpu

DELTA = 4e-5
OUT = 1.1e-4


def make(b, hkv, hq, n, d, seed=0, nmax=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nmax = n if nmax is None else nmax
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return LQ.Bf16Cache(mk(b, hkv, nmax, d), mk(b, hkv, nmax, d), hq), mk(b, hq, d), g


def reference(cache, q, starts, lens, other, scale=None):
    """out, lse, weights [B][Hkv][Nmax] and sum p |v| in fp64."""
    B, Hq, D = q.shape
    G = Hq // cache.Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros(B, cache.Hkv, cache.Nmax, dtype=torch.float64, device="cuda")
    for b in range(B):
        lo, hi = starts[b], max(starts[b], lens[b])
        for hq in range(Hq):
            k, v = cache.k[b, hq // G, lo:hi].double(), cache.v[b, hq // G, lo:hi].double()
            s = scale * (k @ q[b, hq].double())
            l = torch.logsumexp(s, 0) if hi > lo else torch.tensor(-math.inf, dtype=torch.float64, device="cuda")
            joint = l if other is None else torch.logaddexp(l, other[1][b, hq].double())
            lse[b, hq] = joint
            if joint == -math.inf:
                continue
            p = torch.exp(s - joint)
            out[b, hq], mag[b, hq] = p @ v, p @ v.abs()
            if other is not None and other[1][b, hq] > -math.inf:
                po = torch.exp(other[1][b, hq].double() - joint)
                out[b, hq] += po * other[0][b, hq].double()
                mag[b, hq] += po * other[0][b, hq].double().abs()
            w[b, hq // G, lo:hi] += p
    return out, lse, w, mag


def check(got, ref, score_in, score_before, starts, lens):
    out, lse, score = got
    ro, rl, w, mag = ref
    assert ((out.double() - ro).abs() <= OUT * mag + 1e-30).all()
    empty = rl == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    assert ((lse.double() - rl)[~empty].abs() <= DELTA).all()
    n = torch.arange(score.shape[2], device="cuda")
    lo, hi = torch.tensor(starts, device="cuda")[:, None, None], torch.tensor(lens, device="cuda")[:, None, None]
    there = ((n >= lo) & (n < hi)).expand_as(score)
    want = score_in.double() + w
    tol = 2 * DELTA * w + 2.0 ** -23 * want.abs()
    assert ((score.double() - want).abs() <= tol)[there].all()
    assert torch.equal(score[~there], score_before[~there])          # other tokens' scores stay


@pytest.mark.parametrize("hkv,hq,d", [(2, 2, 128), (1, 2, 128), (2, 8, 128), (1, 8, 64), (3, 3, 64)])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 257, 2049, 5000])
def test_scored_decode(hkv, hq, d, n):
    b = 3
    cache, q, g = make(b, hkv, hq, n, d, seed=n, nmax=n + 3)
    lens = [n, n // 2, 0]
    starts = [0, n // 5, 0]
    other = (torch.randn(b, hq, d, generator=g, device="cuda"), 2 * torch.randn(b, hq, generator=g, device="cuda"))
    other[1][0, 0] = -math.inf
    other[0][0, 0] = 0
    score = torch.rand(b, hkv, n + 3, generator=g, device="cuda")
    for oth in (None, other):
        before = torch.full_like(score, 7.0)
        got = LQ.bf16_decode_attn_scored(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, score,
                                         score_out=before.clone(), other=oth,
                                         starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        check(got, reference(cache, q, starts, lens, oth), score, before, starts, lens)


def test_scored_decode_in_place_without_scores_and_repeated():
    cache, q, g = make(2, 2, 8, 700, 128)
    lens = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    zeros = torch.zeros(2, 2, 700, device="cuda")
    o1, l1, s1 = LQ.bf16_decode_attn_scored(cache, q, lens, 700, None, score_out=torch.zeros_like(zeros))
    o2, l2, s2 = LQ.bf16_decode_attn_scored(cache, q, lens, 700, zeros)
    assert s2 is zeros and torch.equal(s1, s2) and torch.equal(o1, o2) and torch.equal(l1, l2)
    total = s1.sum((1, 2))
    assert (total - 8).abs().max() <= 8 * 2 * DELTA                  # every query head shares out a weight of one
    ref, lref = LQ.bf16_decode_attn(cache, q, lens, 700)
    assert torch.allclose(o1, ref, rtol=0, atol=1e-5) and torch.allclose(l1, lref, rtol=0, atol=1e-5)
    s3 = s2.clone()
    LQ.bf16_decode_attn_scored(cache, q, lens, 700, s3, out=o2)
    assert torch.allclose(s3, 2 * s1, rtol=1e-6, atol=0)


@pytest.mark.parametrize("hq,n", [(2, 300), (4, 300), (2, 1500), (4, 1500)])
def test_scored_decode_does_not_read_masked_values(hq, n):
    """Infinities and NaN in the slots before the start and behind the length change nothing (one launch, the split
    kernel, the tensor cores)."""
    cache, q, _ = make(2, 2, hq, n, 64, nmax=n + 4)
    starts, lens = [5, 66], [n - 3, 131]
    args = dict(starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    zeros = torch.zeros(2, 2, n + 4, device="cuda")
    clean = LQ.bf16_decode_attn_scored(cache, q, ln, n, None, score_out=zeros.clone(), **args)
    for b in range(2):
        for x in (cache.k, cache.v):
            x[b, :, :starts[b]] = math.nan
            x[b, :, lens[b]:] = math.inf
    dirty = LQ.bf16_decode_attn_scored(cache, q, ln, n, None, score_out=zeros.clone(), **args)
    for x, y in zip(clean, dirty):
        assert torch.equal(x, y)


@pytest.mark.parametrize("b,hkv,hq,n", [(40, 4, 16, 900), (40, 4, 4, 900), (7, 2, 16, 6000), (150, 1, 2, 1100)])
def test_scored_decode_of_ragged_batches(b, hkv, hq, n):
    """More (sequence, KV head) pairs than SMs, pieces that end inside a sequence, sequences without tokens."""
    cache, q, g = make(b, hkv, hq, n, 64, seed=b)
    lens = [(i * 7919 * n // 10007) % (n + 1) if i % 5 else 0 for i in range(b)]
    lens[1], lens[-1] = n, 1
    starts = [0] * b
    score = torch.rand(b, hkv, n, generator=g, device="cuda")
    got = LQ.bf16_decode_attn_scored(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, score,
                                     score_out=torch.zeros_like(score))
    check(got, reference(cache, q, starts, lens, None), score, torch.zeros_like(score), starts, lens)
    for _ in range(3):                                               # equal inputs give equal bits
        again = LQ.bf16_decode_attn_scored(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, score,
                                           score_out=torch.zeros_like(score))
        assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("hq,n", [(2, 300), (8, 300), (2, 1500), (8, 1500)])
def test_scored_decode_does_not_lose_nan(hq, n):
    """A query or another part of NaN makes its row and its KV head's scores NaN and changes nothing else."""
    cache, q, g = make(3, 2, hq, n, 64, seed=12)
    lens = torch.tensor([n, n - 7, 0], dtype=torch.int32, device="cuda")
    other = torch.randn(3, hq, 64, generator=g, device="cuda"), torch.randn(3, hq, generator=g, device="cuda")
    bad_q, bad_o = q.clone(), (other[0], other[1].clone())
    bad_q[1, 0, 7] = math.nan
    bad_o[1][0, hq - 1], bad_o[1][2, 0] = math.nan, math.nan
    call = lambda x, o: LQ.bf16_decode_attn_scored(cache, x, lens, n, None, other=o,  # noqa: E731
                                                   score_out=torch.zeros(3, 2, n, device="cuda"))
    for x, o, rows, heads in ((bad_q, None, [(1, 0)], [(1, 0)]), (q, bad_o, [(0, hq - 1), (2, 0)], [(0, 1)])):
        good, bad = call(q, None if o is None else other), call(x, o)
        row, head = torch.zeros(3, hq, dtype=torch.bool, device="cuda"), torch.zeros(3, 2, n, dtype=torch.bool, device="cuda")
        for at in rows:
            row[at] = True
        for b, h in heads:
            head[b, h, :int(lens[b])] = True
        assert bad[0][row].isnan().all() and bad[1][row].isnan().all() and bad[2][head].isnan().all()
        assert all(torch.equal(u[~m], w[~m]) for u, w, m in zip(good, bad, (row, row, head)))


def test_scored_decode_with_far_scores():
    """Scores that leave the first tokens' reference by more than the exponent's range."""
    for n in (600, 3000):
        cache, q, g = make(1, 1, 2, n, 64, seed=3)
        q[:] = 1
        cache.k[:] = 0
        cache.k[0, 0, :, 0] = torch.linspace(-3000, 3000, n, device="cuda").bfloat16()   # scores to +- 375
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        out, lse, score = LQ.bf16_decode_attn_scored(cache, q, lens, n, None, score_out=torch.zeros(1, 1, n, device="cuda"))
        ro, rl, w, mag = reference(cache, q, [0], [n], None)
        # exact products (one term each): what is left is the exponent, 375 log2(e) at 2^-24 each of a few roundings
        assert ((lse.double() - rl).abs() <= 4 * 2.0 ** -23 * 375).all()
        assert ((out.double() - ro).abs() <= 1e-3 * mag + 1e-30).all()
        assert ((score.double() - w).abs() <= 1e-3 * w + 1e-30).all()


@pytest.mark.parametrize("n", [700, 1500])
def test_scored_decode_reports_a_wait_that_runs_out(n):
    cache, q, _ = make(2, 2, 4, n, 64)
    lens = torch.tensor([n, n // 2], dtype=torch.int32, device="cuda")
    call = lambda: LQ.bf16_decode_attn_scored(cache, q, lens, n, None, score_out=torch.zeros(2, 2, n, device="cuda"))  # noqa: E731
    good = call()
    LQ.fault_check()
    before = LQ.wait_limit_ns()
    LQ.set_wait_limit_ns(0)
    try:
        bad = call()
        with pytest.raises(LQ.LoopVQError) as e:
            LQ.fault_check()
        assert e.value.status == 5
        assert bad[0].isnan().all() and bad[1].isnan().all()
    finally:
        LQ.set_wait_limit_ns(before)
    again = call()
    LQ.fault_check()
    assert all(torch.equal(x, y) for x, y in zip(good, again))


def evict_reference(k, v, score, pos, lens, next_pos, budget, n_sink, n_recent):
    """Row by row on the host: what slot every kept token ends in."""
    k, v, score, pos = k.clone(), v.clone(), score.clone(), pos.clone()
    B, H = score.shape[:2]
    for b in range(B):
        n = int(lens[b])
        if n <= budget:
            continue
        for h in range(H):
            p, s = pos[b, h, :n].tolist(), score[b, h, :n].tolist()

            def rank(i):
                if p[i] < n_sink or p[i] >= int(next_pos[b]) - n_recent:
                    return (0, 0.0, i)
                return (2, 0.0, i) if s[i] != s[i] else (1, -s[i], i)

            kept = set(sorted(range(n), key=rank)[:budget])
            holes = [i for i in range(budget) if i not in kept]
            sources = sorted(i for i in kept if i >= budget)
            assert len(holes) == len(sources)
            if holes:
                for x in (k, v, score, pos):
                    x[b, h, holes] = x[b, h, sources]
    return k, v, score, pos, [min(int(n), budget) for n in lens]


def run_evict(b, hkv, d, nmax, lens, budget, n_sink, n_recent, in_place, scores="skewed", seed=0, max_len=None):
    cache, _, g = make(b, hkv, hkv, nmax, d, seed=seed)
    score = torch.exp(2 * torch.randn(b, hkv, nmax, generator=g, device="cuda"))
    if scores == "ties":
        score = (score * 2).floor() / 2
    elif scores == "equal":
        score = torch.ones_like(score)
    elif scores == "odd":
        score[..., ::3] = -math.inf
        score[..., 1::5] = math.nan
        score[..., 2::7] = math.inf
        score[..., 3::11] *= -1
        score[..., 4::13] = -0.0
        score[..., 5::13] = 0.0
    pos = torch.rand(b, hkv, nmax, generator=g, device="cuda").argsort(2).int()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    next_pos = torch.full((b,), nmax, dtype=torch.int32, device="cuda")
    want = evict_reference(cache.k.cpu(), cache.v.cpu(), score.cpu(), pos.cpu(), lens, next_pos.cpu(), budget, n_sink,
                           n_recent)
    kept = dict() if in_place else dict(score_out=torch.full_like(score, 5.0), pos_out=torch.full_like(pos, -3),
                                        lens_out=torch.full_like(lens_t, -7))
    before = (kept.get("score_out", score).clone(), kept.get("pos_out", pos).clone())
    so, po, lo = LQ.bf16_evict(cache, score, pos, lens_t, next_pos, nmax if max_len is None else max_len, budget,
                               n_sink, n_recent, **kept)
    torch.cuda.synchronize()
    assert lo.tolist() == want[4]
    assert torch.equal(cache.k.cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(cache.v.cpu().view(torch.int16), want[1].view(torch.int16))
    for i in range(b):
        n = want[4][i]
        assert torch.equal(so[i, :, :n].cpu().view(torch.int32), want[2][i, :, :n].view(torch.int32))
        assert torch.equal(po[i, :, :n].cpu(), want[3][i, :, :n])
        assert torch.equal(so[i, :, n:].view(torch.int32), before[0][i, :, n:].view(torch.int32))
        assert torch.equal(po[i, :, n:], before[1][i, :, n:])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("scores", ["skewed", "ties", "equal", "odd"])
@pytest.mark.parametrize("nmax,budget", [(2, 1), (33, 32), (100, 7), (257, 256), (1030, 500), (5001, 4097)])
def test_evict(nmax, budget, scores, in_place):
    lens = [nmax, max(1, nmax - 1), budget, budget - 1, 0]
    run_evict(5, 2, 64, nmax, lens, budget, min(2, budget // 2), min(3, budget // 2), in_place, scores, seed=nmax)


@pytest.mark.parametrize("n_sink,n_recent,budget", [(0, 0, 40), (40, 0, 40), (0, 40, 40), (8, 32, 40), (0, 0, 1)])
def test_evict_protected_positions(n_sink, n_recent, budget):
    run_evict(2, 3, 128, 200, [200, 150], budget, n_sink, n_recent, False, "ties")


@pytest.mark.parametrize("scores", ["skewed", "ties", "equal"])
@pytest.mark.parametrize("nmax", [1280, 1281, 2560, 2561, 5120, 5121, 10240, 10241, 20480, 20481, 40960, 40961, 60001])
def test_evict_long(nmax, scores):
    """Both sides of the sizes where the selection takes more registers, more CTAs, or its keys from memory again."""
    run_evict(2, 1, 64, nmax, [nmax, nmax - 7], nmax // 3, 8, 64, True, scores)


@pytest.mark.parametrize("hkv,in_place", [(1, True), (8, True), (8, False), (9, True), (16, True), (16, False), (17, True)])
@pytest.mark.parametrize("budget", [1024, 1300, 1700])
def test_evict_few_and_many_rows(hkv, in_place, budget):
    """Steps that one launch does, with clusters of a sequence's heads and without, and those that two do."""
    run_evict(3, hkv, 128, 1800, [1800, budget + 1, budget], budget, 4, 32, in_place, "ties")


def test_evict_equal_positions_and_clamped_lengths():
    """More protected slots than the budget holds: the lowest; a length past max_len counts as max_len."""
    cache, _, g = make(1, 1, 1, 64, 64)
    score = torch.rand(1, 1, 64, generator=g, device="cuda")
    pos = torch.zeros(1, 1, 64, dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    so, po, lo = LQ.bf16_evict(cache, score.clone(), pos, lens, torch.tensor([5], dtype=torch.int32, device="cuda"), 60,
                               10, 8, 2)
    assert lo.tolist() == [10] and torch.equal(so[..., :10], score[..., :10])


def test_decode_evict_steps_together():
    """A run as it is used: append, scored decode, evict, with attention over exactly the kept tokens."""
    b, hkv, hq, d, budget, steps = 2, 2, 4, 64, 96, 40
    nmax = budget + 1
    cache, _, g = make(b, hkv, hq, nmax, d, seed=5)
    score = torch.zeros(b, hkv, nmax, device="cuda")
    pos = torch.zeros(b, hkv, nmax, dtype=torch.int32, device="cuda")
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    all_k, all_v, n = [], [], 0
    for step in range(budget + steps):
        kn, vn = (torch.randn(b, hkv, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        all_k.append(kn)
        all_v.append(vn)
        cache.k[:, :, n], cache.v[:, :, n], pos[:, :, n], score[:, :, n] = kn, vn, step, 0
        lens += 1
        q = torch.randn(b, hq, d, generator=g, device="cuda", dtype=torch.bfloat16)
        out, lse, score = LQ.bf16_decode_attn_scored(cache, q, lens, nmax, score)
        keys, values = torch.stack(all_k, 2), torch.stack(all_v, 2)
        at = pos[:, :, :n + 1].long()[..., None].expand(-1, -1, -1, d)
        assert torch.equal(keys.gather(2, at), cache.k[:, :, :n + 1])
        assert torch.equal(values.gather(2, at), cache.v[:, :, :n + 1])
        if step % 16 == 0 or step > budget + steps - 3:
            ro, rl, _, mag = reference(cache, q, [0] * b, [n + 1] * b, None)
            assert ((out.double() - ro).abs() <= OUT * mag).all()
        LQ.bf16_evict(cache, score, pos, lens, torch.full((b,), step + 1, dtype=torch.int32, device="cuda"), nmax,
                      budget, 4, 16)
        n = min(n + 1, budget)
        assert lens.tolist() == [n] * b
        for i in range(b):
            for h in range(hkv):
                live = sorted(pos[i, h, :n].tolist())
                assert len(set(live)) == n and live[:min(4, n)] == list(range(min(4, n)))
                recent = range(max(0, step + 1 - 16), step + 1)
                assert set(recent) <= set(live)


def test_captured_and_on_another_stream():
    cache, q, g = make(2, 2, 4, 500, 128, seed=9)
    lens = torch.tensor([500, 444], dtype=torch.int32, device="cuda")
    score = torch.rand(2, 2, 500, generator=g, device="cuda")
    pos = torch.arange(500, device="cuda", dtype=torch.int32).expand(2, 2, 500).contiguous()
    nxt = torch.tensor([500, 500], dtype=torch.int32, device="cuda")
    k0, v0 = cache.k.clone(), cache.v.clone()
    eager = LQ.bf16_decode_attn_scored(cache, q, lens, 500, score, score_out=torch.zeros_like(score))
    e2 = LQ.bf16_evict(cache, eager[2], pos, lens, nxt, 500, 100, score_out=torch.zeros_like(score),
                       pos_out=torch.zeros_like(pos), lens_out=torch.zeros_like(lens))
    ke = cache.k.clone()
    cache.k.copy_(k0)
    cache.v.copy_(v0)
    so, so2 = torch.zeros_like(score), torch.zeros_like(score)
    po, lo = torch.zeros_like(pos), torch.zeros_like(lens)
    out, lse = torch.empty_like(eager[0]), torch.empty_like(eager[1])
    w1 = torch.empty(LQ.bf16_scored_workspace_bytes(cache, 500), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(LQ.bf16_evict_workspace_bytes(cache, 500, 100), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        LQ.bf16_decode_attn_scored(cache, q, lens, 500, score, score_out=so, out=out, lse=lse, workspace=w1)
        LQ.bf16_evict(cache, so, pos, lens, nxt, 500, 100, score_out=so2, pos_out=po, lens_out=lo, workspace=w2)
    for _ in range(3):
        cache.k.copy_(k0)
        cache.v.copy_(v0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1]) and torch.equal(so, eager[2])
    assert torch.equal(so2, e2[0]) and torch.equal(po, e2[1]) and torch.equal(lo, e2[2]) and torch.equal(cache.k, ke)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = LQ.bf16_decode_attn_scored(cache, q, lens, 500, score, score_out=torch.zeros_like(score), stream=side,
                                       workspace=w1, out=torch.empty_like(out), lse=torch.empty_like(lse))
    side.synchronize()
    assert again[0].isfinite().all()


@pytest.mark.parametrize("hq,n,budget", [(2, 500, 490), (8, 2100, 300)])
def test_two_sequences_of_calls_at_once(hq, n, budget):
    """Decode and eviction of two caches on two streams, each with workspaces of its own, give what they give alone."""
    sets, alone = [], []
    for seed in (20, 21):
        cache, q, g = make(2, 2, hq, n, 128, seed=seed)
        lens = torch.tensor([n, n - 30], dtype=torch.int32, device="cuda")
        pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(2, 2, n).contiguous()
        score = torch.rand(2, 2, n, generator=g, device="cuda")
        sets.append((cache, q, lens, score, pos))

    def steps(cache, q, lens, score, pos, stream):
        out = torch.empty(2, hq, 128, device="cuda"), torch.empty(2, hq, device="cuda")
        ws = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in
              (LQ.bf16_scored_workspace_bytes(cache, n), LQ.bf16_evict_workspace_bytes(cache, n, budget))]
        nxt = torch.full((2,), n, dtype=torch.int32, device="cuda")
        yield
        for _ in range(6):
            LQ.bf16_decode_attn_scored(cache, q, lens, n, score, score_out=score, out=out[0], lse=out[1], workspace=ws[0],
                                       stream=stream)
            LQ.bf16_evict(cache, score, pos, lens, nxt, n, budget, n_sink=4, n_recent=16, score_out=score, pos_out=pos,
                          lens_out=lens, workspace=ws[1], stream=stream)
            yield
        yield out + (lens, score[..., :budget], pos[..., :budget], cache.k[:, :, :budget], cache.v[:, :, :budget])

    def copy(cache, *rest):
        return (LQ.Bf16Cache(cache.k.clone(), cache.v.clone(), hq),) + tuple(x.clone() for x in rest)

    for x in sets:
        alone.append(list(steps(*copy(*x), None))[-1])
    streams = [torch.cuda.Stream() for _ in sets]
    runs = [steps(*copy(*x), s) for x, s in zip(sets, streams)]
    for r in runs:
        next(r)
    torch.cuda.synchronize()
    for _ in range(6):
        for r in runs:
            next(r)
    torch.cuda.synchronize()
    for r, want in zip(runs, alone):
        assert all(torch.equal(x, y) for x, y in zip(next(r), want))
    LQ.fault_check()
