"""Edges of the shared-prefix, scored and evicting calls that a user's program can reach: full lists, scores of -inf, long
runs of accumulation, default workspaces on other streams, calls in a row without a kernel of another library between."""
import math

import pytest
import torch

import looped_lm_decode_b200 as LQ
from tests.test_gpu_evict import evict_reference

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ eviction

@pytest.mark.parametrize("count", [509, 510, 511, 512])
@pytest.mark.parametrize("own", [0, 1, 2, 100, 300])
@pytest.mark.parametrize("need", [1, 300, 508])
def test_evict_with_a_full_list(count, own, need):
    """The bin of the threshold holds as many keys as are ranked directly, all but `own` of them in the first of the row's
    two CTAs: places at the end of the list."""
    n, split, budget = 5000, 2560, 700
    g = gen(count * 7 + own)
    at = torch.cat([torch.randperm(split, generator=g, device="cuda")[:count - own],
                    split + torch.randperm(n - split, generator=g, device="cuda")[:own]])
    score = torch.full((n,), 0.125, device="cuda")
    free = torch.ones(n, dtype=torch.bool, device="cuda")
    free[at] = False
    rest = torch.nonzero(free).view(-1)
    score[rest[torch.randperm(len(rest), generator=g, device="cuda")[:budget - need]]] = 8.0
    score[at] = 1 + torch.randint(0, 1000, (count,), generator=g, device="cuda") / 4096     # one bin, some of them equal
    score = score.view(1, 1, n)
    cache = LQ.Bf16Cache(bf16(g, 1, 1, n, 64), bf16(g, 1, 1, n, 64), 1)
    pos = torch.arange(n, device="cuda", dtype=torch.int32).view(1, 1, n)
    want = evict_reference(cache.k.cpu(), cache.v.cpu(), score.cpu(), pos.cpu(), [n], torch.tensor([n]), budget, 0, 0)
    so, po, lo = LQ.bf16_evict(cache, score, pos, i32([n]), i32([n]), n, budget, n_sink=0, n_recent=0)
    assert lo.tolist() == [budget]
    assert torch.equal(so[..., :budget].cpu(), want[2][..., :budget]) and torch.equal(po[..., :budget].cpu(), want[3][..., :budget])
    assert torch.equal(cache.k.cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(cache.v.cpu().view(torch.int16), want[1].view(torch.int16))


@pytest.mark.parametrize("hkv", [3, 16, 17])
def test_evict_with_one_array_of_lengths_and_positions(hkv):
    """The next position is the length, in one array that the call shortens."""
    n, budget, b = 900, 800, 6
    g = gen(hkv)
    cache = LQ.Bf16Cache(bf16(g, b, hkv, n, 64), bf16(g, b, hkv, n, 64), hkv)
    score = torch.rand(b, hkv, n, generator=g, device="cuda")
    pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(b, hkv, n).contiguous()
    lens = i32([900, 850, 801, 800, 12, 0])
    want = evict_reference(cache.k.cpu(), cache.v.cpu(), score.cpu(), pos.cpu(), lens.tolist(), lens.cpu(), budget, 8, 64)
    LQ.bf16_evict(cache, score, pos, lens, lens, n, budget)
    assert lens.tolist() == want[4] and torch.equal(cache.k.cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(pos.cpu()[..., :12], want[3][..., :12])


# ------------------------------------------------------------------ streams

def coded_cache(g, hkv, hq, d, c, tc, entries, nmax, layers=1, loops=4, seqs=1):
    cache = LQ.Cache(layers, loops, tc, hkv, hq, d, c, entries, seqs, nmax)
    cache.codebook.copy_(bf16(g, cache.codebook.numel()).view(torch.int16))
    LQ.prepare(cache)
    cache.idx.copy_(torch.randint(-2 ** 31, 2 ** 31, cache.idx.shape, generator=g, device="cuda", dtype=torch.int64).int())
    return cache


def test_default_memory_on_two_streams():
    """Calls that bring no memory of their own, in turn on the current stream and another without a wait between: each
    gives what it gives alone."""
    g = gen(30)
    n, hkv, hq, rows = 20000, 4, 16, 48
    cache = LQ.Bf16Cache(bf16(g, 2, hkv, n, 128), bf16(g, 2, hkv, n, 128), hq)
    coded = coded_cache(g, hkv, hq, 128, 8, 4, 256, n)
    q, qb, lens = bf16(g, rows, hq, 128), bf16(g, 2, hq, 128), i32([n, n - 7])
    score = torch.rand(2, hkv, n, generator=g, device="cuda")
    outs = [torch.zeros_like(score) for _ in range(16)]
    calls = (lambda s, i: LQ.bf16_shared_attn(cache, 0, q, lens, n, stream=s),
             lambda s, i: LQ.shared_attn(coded, 0, 1, 0, q, lens[:1], n, stream=s),
             lambda s, i: LQ.bf16_decode_attn_scored(cache, qb, lens, n, score, score_out=outs[i], stream=s)[:2])
    side = torch.cuda.Stream()
    for call in calls:
        want = [x.clone() for x in call(None, 0)]
        torch.cuda.synchronize()
        got = [call(side if i % 2 else None, i) for i in range(16)]
        torch.cuda.synchronize()
        LQ.fault_check()
        assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))
        del got
    k, v, pos = cache.k.clone(), cache.v.clone(), torch.arange(n, device="cuda", dtype=torch.int32).expand(2, hkv, n).contiguous()
    both = [LQ.Bf16Cache(k.clone(), v.clone(), hq) for _ in range(2)]
    res = [[torch.zeros_like(score), torch.zeros_like(pos), torch.zeros_like(lens)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):                                               # workspaces of 2 x 4 x 12001 words
        x = res[i % 2]
        LQ.bf16_evict(both[i % 2], score, pos, lens, lens, n, 6000, score_out=x[0], pos_out=x[1], lens_out=x[2],
                      stream=side if i % 2 else None)
        if i < 2:                                                    # (kept rows move on from call to call)
            torch.cuda.synchronize()
            first = [y.clone() for y in res[i]] + [both[i].k.clone()]
            keep = first if i == 0 else keep
            assert all(torch.equal(y, z) for y, z in zip(first, keep))
    torch.cuda.synchronize()
    assert all(torch.equal(y, z) for y, z in zip(res[0], res[1])) and torch.equal(both[0].k, both[1].k)


def test_a_stream_of_another_gpu_is_refused():
    class Stream:
        device, cuda_stream = torch.device("cuda", torch.cuda.current_device() + 1), 0

    g = gen(31)
    cache = LQ.Bf16Cache(bf16(g, 1, 1, 64, 64), bf16(g, 1, 1, 64, 64), 1)
    with pytest.raises(LQ.LoopVQError) as e:
        LQ.bf16_shared_attn(cache, 0, bf16(g, 1, 1, 64), i32([64]), 64, stream=Stream())
    assert e.value.status == 1


def test_default_memory_of_decode_and_merge_on_two_streams():
    g = gen(32)
    n, hkv, hq = 20000, 4, 16
    cache = LQ.Bf16Cache(bf16(g, 2, hkv, n, 128), bf16(g, 2, hkv, n, 128), hq)
    coded = coded_cache(g, hkv, hq, 128, 8, 4, 256, n, seqs=2)
    q, lens = bf16(g, 2, hq, 128), i32([n, n - 7])
    part = torch.randn(2, hq, 128, generator=g, device="cuda"), torch.randn(2, hq, generator=g, device="cuda")
    side = torch.cuda.Stream()
    for call in (lambda s: LQ.bf16_decode_attn(cache, q, lens, n, stream=s), lambda s: LQ.decode_attn(coded, 0, 1, q, lens, n, stream=s),
                 lambda s: LQ.merge2(*part, *part, stream=s)):
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        got = [call(side if i % 2 else None) for i in range(16)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))


# ------------------------------------------------------------------ calls in a row

@pytest.mark.parametrize("hkv,hq", [(2, 2), (2, 8), (8, 8)])
@pytest.mark.parametrize("n", [900, 2400])
def test_lengths_that_an_eviction_writes_are_read_by_the_next_call(n, hkv, hq):
    """Evictions in place with scored decodes, prefix attentions and further evictions right behind them, in a graph without
    a kernel of anything else between: what the same calls give one by one."""
    b, d, steps = 4, 64, 12
    g = gen(n + hkv)
    k, v, q = bf16(g, b, hkv, n, d), bf16(g, b, hkv, n, d), bf16(g, b, hq, d)
    score0 = torch.rand(b, hkv, n, generator=g, device="cuda")
    pos0 = torch.arange(n, device="cuda", dtype=torch.int32).expand(b, hkv, n).contiguous()
    lens0, nxt = i32([n, n - 5, n - 60, n - 200]), i32([n] * b)
    budgets = [n - 10 - 20 * i for i in range(steps)]

    def run(cache, score, pos, lens, out, lse, ws, wait):
        for i, budget in enumerate(budgets):
            LQ.bf16_evict(cache, score, pos, lens, nxt, n, budget, n_sink=4, n_recent=16, workspace=ws[0])
            wait()
            if i % 3 == 0:
                LQ.bf16_decode_attn_scored(cache, q, lens, n, score, out=out[i], lse=lse[i], workspace=ws[1])
            elif i % 3 == 1:
                LQ.bf16_shared_attn(cache, 1, q, lens, n, out=out[i], lse=lse[i], workspace=ws[2])
            wait()

    def fresh():
        cache = LQ.Bf16Cache(k.clone(), v.clone(), hq)
        need = [max(LQ.bf16_evict_workspace_bytes(cache, n, x) for x in budgets), LQ.bf16_scored_workspace_bytes(cache, n),
                LQ.bf16_shared_workspace_bytes(cache, b, n)]
        return (cache, score0.clone(), pos0.clone(), lens0.clone(), torch.zeros(steps, b, hq, d, device="cuda"),
                torch.zeros(steps, b, hq, device="cuda"), [torch.zeros(x, dtype=torch.uint8, device="cuda") for x in need])

    alone = fresh()
    run(*alone, torch.cuda.synchronize)
    assert alone[3].tolist() == [budgets[-1]] * b
    for _ in range(3):
        state = fresh()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run(*state, lambda: None)
        graph.replay()
        torch.cuda.synchronize()
        LQ.fault_check()
        m = budgets[-1]
        assert torch.equal(state[3], alone[3]) and torch.equal(state[4], alone[4]) and torch.equal(state[5], alone[5])
        assert torch.equal(state[1][..., :m], alone[1][..., :m]) and torch.equal(state[2][..., :m], alone[2][..., :m])
        assert torch.equal(state[0].k[:, :, :m], alone[0].k[:, :, :m]) and torch.equal(state[0].v[:, :, :m], alone[0].v[:, :, :m])


# ------------------------------------------------------------------ scores of -inf and of the lowest values
#
# Tolerances.  A score is a sum over D products; here one of them moves it by FAR natural units, so the sum's roundings (8 of
# 2^-22 of sum |q k| scale, as in test_gpu_shared.py, where that sum is below 8) grow by (8 + FAR) / 8, and weights and
# outputs with them: GROW times that file's bounds.

FAR = 100.0
GROW = 1 + FAR / 8
LOWEST = torch.finfo(torch.bfloat16).min


def masked_case(g, b, hkv, hq, n, d, masked, kind):
    """Caches and queries whose tokens `masked` score -inf (or about -1e37), and all others FAR below 0: beyond fp32's exponent
    range from a reference of 0."""
    k, v, q = bf16(g, b, hkv, n, d), bf16(g, b, hkv, n, d), bf16(g, b, hq, d)
    q[..., 1], k[..., 1] = 8, -FAR * math.sqrt(d) / 8
    q[..., 0], k[..., 0] = (1, 0) if kind == "inf" else (0.5, 0)
    k[:, :, masked, 0] = -math.inf if kind == "inf" else LOWEST
    return k, v, q


def fp64_attention(q, k, v, other=None):
    """q [Hq][D], k and v [Hkv][n][D] of one sequence: out, lse, sum p |v| and every token's weight per KV head.  Scores past
    fp32's range are -inf."""
    hkv, d = k.shape[0], q.shape[-1]
    s = torch.einsum("hgd,hnd->hgn", q.double().view(hkv, -1, d), k.double()) / math.sqrt(d)
    s = torch.where(s < torch.finfo(torch.float32).min, -math.inf, s)
    lse = torch.logsumexp(s, 2)
    joint = lse if other is None else torch.logaddexp(lse, other[1].double().view(hkv, -1))
    p = torch.exp(s - torch.where(joint == -math.inf, 0.0, joint)[..., None])
    out, mag = p @ v.double(), p @ v.double().abs()
    if other is not None:
        po = torch.exp(other[1].double().view(hkv, -1) - torch.where(joint == -math.inf, 0.0, joint))[..., None]
        out, mag = out + po * other[0].double().view(hkv, -1, d), mag + po * other[0].double().abs().view(hkv, -1, d)
    return out.reshape(-1, d), joint.reshape(-1), mag.reshape(-1, d), p.sum(1)


def close(out, lse, want):
    ro, rl, mag = want[:3]
    empty = rl == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    assert ((out.double() - ro).abs() <= GROW * 2.5e-4 * mag).all(), ((out.double() - ro).abs() / (mag + 1e-30)).max().item()
    assert ((lse.double() - rl)[~empty].abs() <= GROW * 1e-4).all()


def spots(which, n):
    return dict(first=slice(0, 1), tiles=slice(0, min(n - 1, 300)), every_other=slice(0, n, 2), all=slice(0, n))[which]


@pytest.mark.parametrize("kind", ["inf", "lowest"])
@pytest.mark.parametrize("which", ["first", "tiles", "every_other", "all"])
@pytest.mark.parametrize("n", [200, 900, 5000])
@pytest.mark.parametrize("rows,hkv,hq", [(1, 1, 1), (5, 2, 8), (60, 2, 4), (300, 1, 1)])
def test_prefix_scores_of_minus_infinity_weigh_nothing(rows, hkv, hq, n, which, kind):
    """At the first tokens above all, which give some kernels their reference: the other tokens are not lost."""
    if kind == "lowest" and which == "all":
        pytest.skip("rounding decides among scores of -1e37: test_prefix_scores_far_from_zero")
    g, d = gen(rows + n), 128
    k, v, _ = masked_case(g, 1, hkv, hq, n, d, spots(which, n), kind)
    q = bf16(g, rows, hq, d)
    q[..., 1], q[..., 0] = 8, 1 if kind == "inf" else 0.5
    cache = LQ.Bf16Cache(k, v, hq)
    other = torch.randn(rows, hq, d, generator=g, device="cuda"), torch.randn(rows, hq, generator=g, device="cuda") - FAR
    for o in (None, other):
        out, lse = LQ.bf16_shared_attn(cache, 0, q, i32([n]), n, other=o)
        LQ.fault_check()
        for r in range(0, rows, 7):
            close(out[r], lse[r], fp64_attention(q[r], k[0], v[0], None if o is None else (o[0][r], o[1][r])))


@pytest.mark.parametrize("kind", ["inf", "lowest"])
@pytest.mark.parametrize("which", ["first", "tiles", "every_other"])
@pytest.mark.parametrize("hq,n", [(2, 300), (8, 300), (4, 1500), (8, 5000)])
def test_scored_decode_with_scores_of_minus_infinity(hq, n, which, kind):
    """On the tensor cores, in one launch and in two: outputs, log-sum-exps and weights."""
    g, b, hkv, d = gen(n + hq), 3, 2, 64
    k, v, q = masked_case(g, b, hkv, hq, n, d, spots(which, n), kind)
    score = torch.rand(b, hkv, n, generator=g, device="cuda")
    other = torch.randn(b, hq, d, generator=g, device="cuda"), torch.randn(b, hq, generator=g, device="cuda") - FAR
    for o in (None, other):
        out, lse, s = LQ.bf16_decode_attn_scored(LQ.Bf16Cache(k, v, hq), q, i32([n] * b), n, score, other=o,
                                                 score_out=torch.zeros_like(score))
        LQ.fault_check()
        for i in range(b):
            want = fp64_attention(q[i], k[i], v[i], None if o is None else (o[0][i], o[1][i]))
            close(out[i], lse[i], want)
            total = score[i].double() + want[3]
            assert ((s[i].double() - total).abs() <= GROW * 2e-4 * want[3] + 2.0 ** -23 * total).all()


@pytest.mark.parametrize("rows,n", [(4, 200), (4, 900), (4, 5000), (60, 300), (60, 5000), (300, 300), (300, 5000)])
def test_prefix_scores_far_from_zero(rows, n):
    """Every score about -1e37, or one of 1e37: whatever rounding leaves of their order, a row is an average of values, or the
    one value, and its log-sum-exp the scores' size."""
    g, d = gen(rows + n), 128
    k, v, q = bf16(g, 1, 1, n, d), bf16(g, 1, 1, n, d), bf16(g, rows, 1, d)
    q[..., 0], size = 0.5, -0.5 * LOWEST / math.sqrt(d)
    for keys, sign in ((slice(0, n), -1), (slice(n // 2, n // 2 + 1), 1), (slice(n - 1, n), 1), (slice(0, 1), 1)):
        kk = k.clone()
        kk[0, 0, keys, 0] = -LOWEST * sign
        out, lse = LQ.bf16_shared_attn(LQ.Bf16Cache(kk, v, 1), 0, q, i32([n]), n)
        LQ.fault_check()
        assert ((lse / (sign * size) - 1).abs() <= 2.0 ** -20).all()
        if sign < 0:
            assert (out <= v.float().amax(2) + 1e-4).all() and (out >= v.float().amin(2) - 1e-4).all()
        else:
            assert torch.equal(out[:, 0], v[0, 0, keys].float().expand(rows, d))


@pytest.mark.parametrize("hq,n", [(1, 300), (8, 300), (1, 1500), (4, 1500), (8, 5000)])
def test_scored_decode_with_scores_far_from_zero(hq, n):
    g, b, d = gen(hq + n), 2, 64
    k, v, q = bf16(g, b, 1, n, d), bf16(g, b, 1, n, d), bf16(g, b, hq, d)
    q[..., 0] = 0.5
    for at in (0, n // 2, n - 1):
        kk = k.clone()
        kk[:, 0, at, 0] = -LOWEST
        out, lse, score = LQ.bf16_decode_attn_scored(LQ.Bf16Cache(kk, v, hq), q, i32([n] * b), n, None,
                                                     score_out=torch.zeros(b, 1, n, device="cuda"))
        LQ.fault_check()
        assert torch.equal(out, v[:, :, at].float().expand(b, hq, d)) and (score[:, 0, at] == hq).all()
        assert (score.sum(2) == hq).all() and ((lse / (-0.5 * LOWEST / math.sqrt(d)) - 1).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("hq,n", [(2, 300), (8, 300), (4, 1500), (8, 5000)])
def test_heads_whose_every_score_is_minus_infinity_weigh_nothing(hq, n):
    """Beside heads of the same KV head that have weight: no output, a log-sum-exp of -inf (or the other part's), and no trace
    in the scores.  A KV head of nothing but such heads leaves its scores as they were."""
    g, b, hkv, d = gen(n + hq), 2, 2, 64
    k, v, q = bf16(g, b, hkv, n, d), bf16(g, b, hkv, n, d), bf16(g, b, hq, d)
    k[..., 0], q[..., 0] = LOWEST, 2.0 ** -126                       # adds about -4 to an ordinary head's sums
    q[0, 0, 0], q[1, hq // 2:, 0] = 64, 64                           # overflows to -inf: one head; a KV head's all
    score = torch.rand(b, hkv, n, generator=g, device="cuda")
    other = torch.randn(b, hq, d, generator=g, device="cuda"), torch.randn(b, hq, generator=g, device="cuda")
    for o in (None, other):
        out, lse, s = LQ.bf16_decode_attn_scored(LQ.Bf16Cache(k, v, hq), q, i32([n] * b), n, score, other=o,
                                                 score_out=torch.zeros_like(score))
        LQ.fault_check()
        for i in range(b):
            want = fp64_attention(q[i], k[i], v[i], None if o is None else (o[0][i], o[1][i]))
            close(out[i], lse[i], want)
            total = score[i].double() + want[3]
            assert ((s[i].double() - total).abs() <= GROW * 2e-4 * want[3] + 2.0 ** -23 * total).all()
        assert torch.equal(s[1, 1], score[1, 1])
        if o is not None:
            assert torch.equal(out[0, 0], o[0][0, 0]) and torch.allclose(lse[0, 0], o[1][0, 0], rtol=1e-6, atol=0)


@pytest.mark.parametrize("kind", ["inf", "lowest"])
@pytest.mark.parametrize("which", ["first", "tiles", "every_other", "all"])
@pytest.mark.parametrize("hq,n", [(2, 300), (2, 1500), (2, 9000), (4, 1500), (16, 300)])
def test_decode_with_scores_of_minus_infinity(hq, n, which, kind):
    """The kernel that splits a sequence's tokens: with scores (one head per KV head) and without (any)."""
    if kind == "lowest" and which == "all":
        pytest.skip("rounding decides among scores of -1e37")
    g, b, hkv, d = gen(n + hq), 2, 2, 64
    k, v, q = masked_case(g, b, hkv, hq, n, d, spots(which, n), kind)
    cache, lens, score = LQ.Bf16Cache(k, v, hq), i32([n, n - 1]), torch.rand(b, hkv, n, generator=g, device="cuda")
    out, lse = LQ.bf16_decode_attn(cache, q, lens, n)
    scored = LQ.bf16_decode_attn_scored(cache, q, lens, n, score, score_out=score.clone())
    for i, m in enumerate(lens.tolist()):
        want = fp64_attention(q[i], k[i, :, :m], v[i, :, :m])
        if kind == "lowest" and which == "tiles" and m == n - 1 == 299:
            # nothing but scores of about -2e37 is left, which fp32 holds to 2^101: it cannot tell them apart, fp64 does
            assert out[i].isfinite().all() and scored[0][i].isfinite().all()
            continue
        close(out[i], lse[i], want)
        close(scored[0][i], scored[1][i], want)
        total = score[i, :, :m].double() + want[3]
        assert ((scored[2][i, :, :m].double() - total).abs() <= GROW * 2e-4 * want[3] + 2.0 ** -23 * total).all()


def test_decode_of_nan_queries_as_before():
    """Of nothing but NaN the decode without scores makes zeros and -inf (as it did), the scored one NaN."""
    g, n = gen(40), 3000
    cache = LQ.Bf16Cache(bf16(g, 1, 1, n, 64), bf16(g, 1, 1, n, 64), 1)
    q = bf16(g, 1, 1, 64)
    q[0, 0, 3] = math.nan
    out, lse = LQ.bf16_decode_attn(cache, q, i32([n]), n)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse, score = LQ.bf16_decode_attn_scored(cache, q, i32([n]), n, None, score_out=torch.zeros(1, 1, n, device="cuda"))
    assert out.isnan().all() and lse.isnan().all() and score.isnan().all()


# ------------------------------------------------------------------ sizes and places no other test reaches

def check_rows(out, lse, q, k, v, rows):
    """Rows of out against fp64: q [rows][Hq][D], k and v [Hkv][n][D]."""
    for r in rows:
        want = fp64_attention(q[r], k, v)
        assert ((out[r].double() - want[0]).abs() <= 2.5e-4 * want[2]).all() and ((lse[r].double() - want[1]).abs() <= 1e-4).all()


@pytest.mark.parametrize("rows", [3, 40, 200])
@pytest.mark.parametrize("layer,t", [(0, 0), (1, 6), (2, 3)])
def test_coded_prefix_of_any_layer_and_block(layer, t, rows):
    from tests.test_gpu_shared import rebuild
    g, n, hkv, hq, d = gen(layer), 333, 2, 4, 128
    cache = coded_cache(g, hkv, hq, d, 4, 4, 256, 336, layers=3, loops=8, seqs=3)
    one = LQ.Cache(1, 8, 4, hkv, hq, d, 4, 256, 3, 336)              # that layer alone, for the plain form
    one.idx.copy_(cache.idx.view(3, -1)[layer])
    one.codebook.copy_(cache.codebook.view(3, -1)[layer])
    LQ.prepare(one)
    q, lens = bf16(g, rows, hq, d), i32([5, n, 9])
    out, lse = LQ.shared_attn(cache, layer, t, 1, q, lens, 336, starts=i32([0, 6, 0]))
    LQ.fault_check()
    k, v = rebuild(one, t, 1, 6, n)
    check_rows(out, lse, q, k, v, range(0, rows, 13))


@pytest.mark.parametrize("rows,n", [(2000, 3000), (1025, 130)])
def test_coded_prefix_of_a_prompt(rows, n):
    from tests.test_gpu_shared import rebuild
    g, hkv, hq, d = gen(rows), 2, 2, 128
    cache = coded_cache(g, hkv, hq, d, 8, 4, 256, (n + 3) // 4 * 4)
    q = bf16(g, rows, hq, d)
    out, lse = LQ.shared_attn(cache, 0, 1, 0, q, i32([n]), n)
    LQ.fault_check()
    check_rows(out, lse, q, *rebuild(cache, 1, 0, 0, n), range(0, rows, 97))


def test_as_many_rows_as_a_grid_holds():
    """65000 blocks of 128 rows."""
    g, rows, hq, d, n = gen(60), 1040000, 8, 64, 5
    cache, q = LQ.Bf16Cache(bf16(g, 1, 1, 8, d), bf16(g, 1, 1, 8, d), hq), bf16(g, rows, hq, d)
    out, lse = LQ.bf16_shared_attn(cache, 0, q, i32([n]), n)
    LQ.fault_check()
    check_rows(out, lse, q, cache.k[0, :, :n], cache.v[0, :, :n], [0, 1, 77777, 524287, 524288, rows - 1])
    for a in range(0, rows, 80000):                                  # all of them, in fp32
        s = (q[a:a + 80000].float() @ cache.k[0, 0, :n].float().T) / math.sqrt(d)
        plain = torch.softmax(s, 2) @ cache.v[0, 0, :n].float()
        assert (out[a:a + 80000] - plain).abs().max().item() <= 1e-3


@pytest.mark.parametrize("hq", [18, 36])
def test_offsets_past_two_to_the_31(hq):
    """18 heads of a million tokens: 2.3e9 elements, the last head past 2^31."""
    g, n, hkv, d = gen(61), 1000000, 18, 128
    k, v = (torch.empty(1, hkv, n, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    cache, start, lens = LQ.Bf16Cache(k, v, hq), n - 700, i32([n - 3])
    for rows in (1, 50):
        q = bf16(g, rows, hq, d)
        out, lse = LQ.bf16_shared_attn(cache, 0, q, lens, n, starts=i32([start]))
        LQ.fault_check()
        check_rows(out, lse, q, k[0, :, start:n - 3], v[0, :, start:n - 3], [0, rows - 1])
    score = torch.zeros(1, hkv, n, device="cuda")
    q = bf16(g, 1, hq, d)
    out, lse, score = LQ.bf16_decode_attn_scored(cache, q, lens, n, score, starts=i32([start]))
    LQ.fault_check()
    check_rows(out, lse, q, k[0, :, start:n - 3], v[0, :, start:n - 3], [0])
    w = fp64_attention(q[0], k[0, :, start:n - 3], v[0, :, start:n - 3])[3]
    assert ((score[0, :, start:n - 3].double() - w).abs() <= 2e-4 * w).all()
    assert (score[..., :start] == 0).all() and (score[..., n - 3:] == 0).all()
    # eviction to 4 slots behind which everything lies: the rows of the last head move, too
    pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(1, hkv, n).contiguous()
    best = score[0].topk(4, 1).indices.sort(1).values
    want = [k[0, h, best[h]].clone() for h in range(hkv)]
    so, po, lo = LQ.bf16_evict(cache, score, pos, lens, i32([n]), n, 4, n_sink=0, n_recent=0)
    assert lo.tolist() == [4] and torch.equal(po[0, :, :4].long(), best)
    assert all(torch.equal(k[0, h, :4], want[h]) for h in range(hkv))
